// k_seqconv.hip -- the causal depthwise convolution over tokens: forward,
// backward and the single-token step (conv_causal_*).
//
// p[t][c] = bias[c] + sum_j w[c][j] X[t-K+1+j][c]: K multiply-adds for two
// elements moved, so HBM is the bound (each row read once and written once;
// the backward pass reads x and dy and writes dx).  A thread owns VEC adjacent
// channels and walks a run of consecutive tokens with the last K rows in
// registers, so a row is loaded once per run plus K-1 rows in front of it
// (which the neighbouring run has just read: cache hits).  The row window is
// indexed by token modulo K with the loop unrolled K times, so that no
// register is ever moved.
//
// Threads of a workgroup lie along the channels first (wide, contiguous
// loads), then along runs of tokens; K or more rows are loaded ahead of their use.
//
// Measured at 8 x 2048 x 2048 bf16, K = 4 with SiLU: forward 27.6 us, 4.9 TB/s, the rate
// of a copy of that size; backward 49.6 us, 4.1 TB/s, of which the vector
// instructions take 31 us (SQ_ACTIVE_INST_VALU) and the reduction 4 us.  8 x 4096 x 4096:
// 88.7 us, 6.05 TB/s, and 163 us, 4.9 TB/s.
#include <type_traits>

#include "seq_common.h"

namespace convfwd {
namespace {

constexpr int kThreads = 256;

// Rows loaded together: a multiple of K, at least three.
template <int K> constexpr int kGroup = K >= 3 ? K : 4;

// Row t of X (t may be negative: the carried rows), VEC channels at c.
template <typename T, int VEC, int K>
__device__ __forceinline__ void x_row(const T *x, int64_t ldx, const T *state, int64_t first, int b, int C, int c,
                                      int t, float (&f)[VEC]) {
    if (t >= 0) {
        load_f32<T, VEC>(x + (first + t) * ldx + c, f);
    } else if (K > 1 && state) {
        load_f32<T, VEC>(state + ((int64_t)b * (K - 1) + (K - 1 + t)) * C + c, f);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = 0.f;
    }
}

template <typename T, int VEC, int K>
__device__ __forceinline__ void load_w(const T *w, int c, float (&wf)[K][VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
#pragma unroll
        for (int j = 0; j < K; ++j) {
            float f[1];
            load_f32<T, 1>(w + (int64_t)(c + i) * K + j, f);
            wf[j][i] = f[0];
        }
}

// The last K-1 rows of X, the state after a sequence of `len` tokens.
template <typename T, int VEC, int K>
__device__ __forceinline__ void write_state(const T *x, int64_t ldx, const T *state, T *out, int64_t first, int len,
                                            int b, int C, int c) {
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
        float f[VEC];
        x_row<T, VEC, K>(x, ldx, state, first, b, C, c, len - (K - 1) + i, f);
        store_f32(out + ((int64_t)b * (K - 1) + i) * C + c, f);
    }
}

// Where a thread works: a run of tl tokens of sequence b, VEC channels from c on.
struct Work {
    int b, c, t0, t1, len;
    int64_t first;
    bool any, head;         // any: channels at all; head: the sequence's first run
};

template <int VEC> __device__ __forceinline__ Work get_work(const Seq &s, int64_t block, int per, int bx_log2, int tl) {
    Work k;
    const int by = kThreads >> bx_log2;
    const int tx = threadIdx.x & ((1 << bx_log2) - 1), ty = threadIdx.x >> bx_log2;
    Block at;
    if (!s.off || per == 1) {
        at.b = (int)((unsigned)block / per);
        at.k = (int)((unsigned)block % per);
    } else {
        at = packed_block(s, by * tl, block);
    }
    const int c = ((blockIdx.y << bx_log2) + tx) * VEC;
    k.any = c < s.C;
    k.c = min(c, s.C - VEC);        // the last threads may share channels, with the same results
    k.b = at.b;
    seq_range(s, k.b, k.first, k.len);
    if (at.k < 0) k.len = 0;
    k.t0 = max(at.k, 0) * by * tl + ty * tl;
    k.t1 = min(k.t0 + tl, k.len);
    k.head = at.k == 0 && ty == 0;
    return k;
}

// K rows from p on, in bf16 or fp32 as they are; only the first `there` of them are, and the first row
// stands in for the others, so that loads need no branch.
template <typename T, int VEC, int K, bool ONCE> struct Rows {
    typename Pack<T, VEC>::type v[K];
    __device__ __forceinline__ void load(const T *p, int64_t ld, int there) {
#pragma unroll
        for (int u = 0; u < K; ++u) {
            const T *q = p + (u < there ? u * ld : 0);
            v[u] = ONCE ? load_once<T, VEC>(q) : load_pack<T, VEC>(q);
        }
    }
};

// grid (blocks of tokens, channel blocks)
template <typename T, int VEC, int K, bool SILU, bool ONCE>
__global__ __launch_bounds__(kThreads) void causal_fwd_kernel(Seq s, const T *__restrict__ x, int64_t ldx,
                                                              const T *__restrict__ w, const float *__restrict__ bias,
                                                              const T *__restrict__ state, T *__restrict__ y,
                                                              int64_t ldy, T *__restrict__ state_out, int per,
                                                              int bx_log2, int tl, Fill f) {
    constexpr int U = kGroup<K>;                   // rows loaded together: a multiple of K
    const int block = (int)blockIdx.x - f.blocks;  // the first workgroups fill
    if (block < 0) {
        fill_rows(s, f, (int64_t)blockIdx.x * gridDim.y + blockIdx.y, (int64_t)f.blocks * gridDim.y);
        return;
    }
    const Work k = get_work<VEC>(s, block, per, bx_log2, tl);
    if (!k.any) return;
    if (K > 1 && state_out && k.head) write_state<T, VEC, K>(x, ldx, state, state_out, k.first, k.len, k.b, s.C, k.c);
    if (k.t0 >= k.t1) return;
    const T *xp = x + (k.first + k.t0) * ldx + k.c;
    T *yp = y + (k.first + k.t0) * ldy + k.c;
    Rows<T, VEC, U, ONCE> next;
    next.load(xp, ldx, k.t1 - k.t0);
    float wf[K][VEC], bf[VEC], win[K][VEC];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) x_row<T, VEC, K>(x, ldx, state, k.first, k.b, s.C, k.c, k.t0 - (K - 1) + j, win[j]);
    load_w<T, VEC, K>(w, k.c, wf);
#pragma unroll
    for (int i = 0; i < VEC; ++i) bf[i] = bias ? bias[k.c + i] : 0.f;
    // at step u (mod K) the new row goes to slot (K-1+u) % K; tap j is slot (u+j) % K
    for (int t = k.t0; t < k.t1; t += U) {
        const Rows<T, VEC, U, ONCE> now = next;
        xp += U * ldx;
        if (t + U < k.t1) next.load(xp, ldx, k.t1 - t - U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            to_f32(now.v[u], win[(K - 1 + u) % K]);
            float p[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                p[i] = bf[i];
#pragma unroll
                for (int j = 0; j < K; ++j) p[i] = fmaf(wf[j][i], win[(u + j) % K][i], p[i]);
                if (SILU) p[i] *= sigmoid(p[i]);
            }
            if (t + u < k.t1) store_f32(yp + u * ldy, p);
        }
        yp += U * ldy;
    }
}

// Backward.  Walking t forward, dp[t] comes from dy[t] and the recomputed p[t];
// row o = t-(K-1) of dX then has all its K terms dp[o..o+K-1].  A run takes
// dw and db from its own tokens and computes the dp of K-1 tokens behind it
// again.  The first run of a sequence also emits rows o < 0, the gradient of
// the carried rows.  Partial sums of dw and db: one row of (K+1) x C floats per
// workgroup, reduced over its runs in LDS in a fixed order, then added over
// workgroups in a fixed order by causal_reduce_kernel.
template <typename T, int VEC, int K, bool SILU, bool ONCE>
__global__ __launch_bounds__(kThreads) void causal_bwd_kernel(Seq s, const T *__restrict__ x, int64_t ldx,
                                                              const T *__restrict__ w, const float *__restrict__ bias,
                                                              const T *__restrict__ state, const T *__restrict__ dy,
                                                              int64_t lddy, T *__restrict__ dx, int64_t lddx,
                                                              T *__restrict__ dstate, float *__restrict__ part,
                                                              int per, int bx_log2, int tl, Fill f) {
    constexpr int U = kGroup<K>;
    __shared__ float red[kThreads * VEC];
    const int block = (int)blockIdx.x - f.blocks;
    if (block < 0) {
        fill_rows(s, f, (int64_t)blockIdx.x * gridDim.y + blockIdx.y, (int64_t)f.blocks * gridDim.y);
        return;
    }
    const int bx = 1 << bx_log2, by = kThreads >> bx_log2;
    const int tx = threadIdx.x & (bx - 1), ty = threadIdx.x >> bx_log2;
    const Work k = get_work<VEC>(s, block, per, bx_log2, tl);
    float dw[K][VEC] = {}, db[VEC] = {};
    const bool head = k.head && K > 1 && dstate;
    if (k.any && (k.t0 < k.t1 || head)) {
        const int end = max(k.t1, k.t0) + K - 1;       // dX rows up to t1 - 1
        const T *xp = x + (k.first + k.t0) * ldx + k.c, *dp_ = dy + (k.first + k.t0) * lddy + k.c;
        Rows<T, VEC, U, ONCE> nx, nd;
        if (k.t0 < k.len) {
            nx.load(xp, ldx, k.len - k.t0);
            nd.load(dp_, lddy, k.len - k.t0);
        }
        float wf[K][VEC], bf[VEC], win[K][VEC], dp[K][VEC];
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) dp[j][i] = win[j][i] = 0.f;
        if (k.t0 < k.t1) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
                x_row<T, VEC, K>(x, ldx, state, k.first, k.b, s.C, k.c, k.t0 - (K - 1) + j, win[j]);
        }
        load_w<T, VEC, K>(w, k.c, wf);
#pragma unroll
        for (int i = 0; i < VEC; ++i) bf[i] = bias ? bias[k.c + i] : 0.f;
        // U rows of a run; inner: all are the run's own and so are the rows of dX that they complete
        const auto group = [&](int t, const Rows<T, VEC, U, ONCE> &x0, const Rows<T, VEC, U, ONCE> &d0, auto inner_) {
            constexpr bool inner = decltype(inner_)::value;
            T *dxp = dx + (k.first + t - (K - 1)) * lddx + k.c;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int tt = t + u;
                float(&d)[VEC] = dp[(K - 1 + u) % K];
                if (inner || tt < k.len) {
                    to_f32(x0.v[u], win[(K - 1 + u) % K]);
                    to_f32(d0.v[u], d);
                    if (SILU) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            float p = bf[i];
#pragma unroll
                            for (int j = 0; j < K; ++j) p = fmaf(wf[j][i], win[(u + j) % K][i], p);
                            const float sg = sigmoid(p);
                            d[i] *= sg * fmaf(p, 1.f - sg, 1.f);
                        }
                    }
                    if (inner || tt < k.t1) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            db[i] += d[i];
#pragma unroll
                            for (int j = 0; j < K; ++j) dw[j][i] = fmaf(d[i], win[(u + j) % K][i], dw[j][i]);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) d[i] = 0.f;
                }
                // dX[o] = sum_j w[j] dp[o+K-1-j], o = tt-K+1: dp[tt-j] is in slot (K-1+u-j) % K.  Tokens in front of
                // the sequence and behind it have no term: an infinite weight must not meet a zero there.
                const int o = tt - (K - 1);
                float g[VEC];
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    const bool there = inner || (tt - j >= 0 && tt - j < k.len);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float dj = dp[(2 * K - 1 + u - j) % K][i], before = j ? g[i] : 0.f;
                        const float sum = j ? fmaf(wf[j][i], dj, before) : wf[j][i] * dj;
                        g[i] = there ? sum : before;
                    }
                }
                if (inner || (o >= k.t0 && o < k.t1))
                    store_f32(dxp + u * lddx, g);
                else if (o < k.t0 && head && tt < K - 1)
                    store_f32(dstate + ((int64_t)k.b * (K - 1) + tt) * s.C + k.c, g);
            }
        };
        for (int t = k.t0; t < end; t += U) {
            const Rows<T, VEC, U, ONCE> x0 = nx, d0 = nd;
            xp += U * ldx;
            dp_ += U * lddy;
            if (t + U < end && t + U < k.len) {
                nx.load(xp, ldx, k.len - t - U);
                nd.load(dp_, lddy, k.len - t - U);
            }
            if (t > k.t0 && t + U <= k.t1)
                group(t, x0, d0, std::true_type{});
            else
                group(t, x0, d0, std::false_type{});
        }
    }
    // the thread of the first run adds its channels over the runs, in order
    for (int j = 0; j <= K; ++j) {
        if (j) __syncthreads();
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            float v = db[i];
#pragma unroll
            for (int q = 0; q < K; ++q) v = j == q ? dw[q][i] : v;
            red[(ty * VEC + i) * bx + tx] = v;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < bx * VEC; e += kThreads) {
            const int q = e & (bx - 1), i = e >> bx_log2, c = ((blockIdx.y << bx_log2) + q) * VEC;
            float v = 0.f;
            for (int r = 0; r < by; ++r) v += red[(r * VEC + i) * bx + q];
            if (c < s.C) part[((int64_t)block * (K + 1) + j) * s.C + min(c, s.C - VEC) + i] = v;
        }
    }
}

// dw (C, K) and db from the workgroups' partial sums: 16 channels of one of the
// K+1 rows per workgroup, 64 strands of partials, each added in order.
__global__ __launch_bounds__(1024) void causal_reduce_kernel(const float *__restrict__ part, int64_t n, int C, int K,
                                                             float *__restrict__ dw, float *__restrict__ db) {
    __shared__ float red[64][17];
    const int cl = threadIdx.x & 15, q = threadIdx.x >> 4, c = blockIdx.x * 16 + cl, j = blockIdx.y;
    float v = 0.f;
    if (c < C)
        for (int64_t i = q; i < n; i += 64) v += part[(i * (K + 1) + j) * C + c];
    red[q][cl] = v;
    __syncthreads();
    if (q < 8) {
        v = 0.f;
        for (int i = 0; i < 8; ++i) v += red[q * 8 + i][cl];
    }
    __syncthreads();
    if (q < 8) red[q][cl] = v;
    __syncthreads();
    if (q == 0 && c < C) {
        v = 0.f;
        for (int i = 0; i < 8; ++i) v += red[i][cl];
        if (j < K)
            dw[(int64_t)c * K + j] = v;
        else if (db)
            db[c] = v;
    }
}

template <typename T, int VEC, int K, bool SILU>
__global__ __launch_bounds__(kThreads) void causal_step_kernel(int B, int C, const T *__restrict__ x, int64_t ldx,
                                                               const T *__restrict__ w, const float *__restrict__ bias,
                                                               T *__restrict__ state, T *__restrict__ y, int64_t ldy) {
    const int per = C / VEC;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (int64_t)B * per) return;
    const int b = (int)(i / per), c = (int)(i % per) * VEC;
    float wf[K][VEC], p[VEC], row[VEC];
    load_w<T, VEC, K>(w, c, wf);
#pragma unroll
    for (int v = 0; v < VEC; ++v) p[v] = bias ? bias[c + v] : 0.f;
    T *sp = state + (int64_t)b * (K - 1) * C + c;
#pragma unroll
    for (int j = 0; j < K; ++j) {
        if (j < K - 1)
            load_f32<T, VEC>(sp + (int64_t)j * C, row);
        else
            load_f32<T, VEC>(x + b * ldx + c, row);
        if (j > 0) store_f32(sp + (int64_t)(j - 1) * C, row);
#pragma unroll
        for (int v = 0; v < VEC; ++v) p[v] = fmaf(wf[j][v], row[v], p[v]);
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v)
        if (SILU) p[v] *= sigmoid(p[v]);
    store_f32(y + b * ldy + c, p);
}

// Channel threads of a workgroup: the power of two that covers the channels,
// 8 to 64.
int channel_log2(int groups) {
    int l = 3;
    while (l < 6 && (1 << l) < groups) ++l;
    return l;
}

struct Tiling {
    int bx_log2, tl, per, cblk;
    int64_t n;              // blocks of tokens
};

// Tokens of a run: long ones read fewer rows twice and leave fewer partial sums, short ones make more
// workgroups.  The longest of 64, 32 and 16 that still gives `least` workgroups: one for each of 256 CUs
// forward (at 8 x 2048 x 2048 bf16, runs of 64, 32, 16: 30.5, 31.3, 33.9 us), two backward, which has
// three waves per SIMD and takes all of them in one round (51, 65, 72 us; 5003 x 999 fp32 packed: 32, 22.6, 21.5).
constexpr int kFwdLeast = 256, kBwdLeast = 512, kShortest = 16;
Tiling tiling(const Seq &s, int vec, int least) {
    Tiling t;
    t.bx_log2 = channel_log2((s.C + vec - 1) / vec);
    t.cblk = (s.C + (vec << t.bx_log2) - 1) / (vec << t.bx_log2);
    for (t.tl = 64;; t.tl >>= 1) {
        const int run = (kThreads >> t.bx_log2) * t.tl;
        t.per = s.T > 0 ? (int)(((int64_t)s.T + run - 1) / run) : 1;
        t.n = block_count(s, run, t.per);
        if (t.tl == kShortest || t.n * t.cblk >= least) return t;
    }
}

template <typename T, int VEC, int K, bool SILU>
void fwd(const Seq &s, const T *x, int64_t ldx, const T *w, const float *bias, const T *state, T *y, int64_t ldy,
         T *state_out, hipStream_t st) {
    const Tiling t = tiling(s, VEC, kFwdLeast);
    const auto run = VEC > 1 && read_once(x, ldx, sizeof(T)) ? causal_fwd_kernel<T, VEC, K, SILU, (VEC > 1)>
                                                             : causal_fwd_kernel<T, VEC, K, SILU, false>;
    const Fill f = fill_of(s, kThreads / 64 * t.cblk, {y}, {ldy});
    run<<<dim3((unsigned)t.n + f.blocks, t.cblk), kThreads, 0, st>>>(s, x, ldx, w, bias, state, y, ldy, state_out, t.per,
                                                                     t.bx_log2, t.tl, f);
}

template <typename T, int VEC, int K, bool SILU>
hipError_t bwd(const Seq &s, const T *x, int64_t ldx, const T *w, const float *bias, const T *state, const T *dy, int64_t lddy,
         T *dx, int64_t lddx, float *dw, float *db, T *dstate, float *part, hipStream_t st) {
    const Tiling t = tiling(s, VEC, kBwdLeast);
    const auto run = VEC > 1 && read_once(x, ldx, sizeof(T)) && read_once(dy, lddy, sizeof(T))
                         ? causal_bwd_kernel<T, VEC, K, SILU, (VEC > 1)> : causal_bwd_kernel<T, VEC, K, SILU, false>;
    const Fill f = fill_of(s, kThreads / 64 * t.cblk, {dx}, {lddx});
    run<<<dim3((unsigned)t.n + f.blocks, t.cblk), kThreads, 0, st>>>(s, x, ldx, w, bias, state, dy, lddy, dx, lddx, dstate, part,
                                                                     t.per, t.bx_log2, t.tl, f);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;              // there are no partial sums
    causal_reduce_kernel<<<dim3((s.C + 15) / 16, K + 1), 1024, 0, st>>>(part, t.n, s.C, K, dw, db);
    return hipGetLastError();
}

template <typename T, int VEC, int K, bool SILU>
void step(const Seq &s, const T *x, int64_t ldx, const T *w, const float *bias, T *state, T *y, int64_t ldy,
          hipStream_t st) {
    const int64_t n = (int64_t)s.B * (s.C / VEC);
    causal_step_kernel<T, VEC, K, SILU><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(
        s.B, s.C, x, ldx, w, bias, state, y, ldy);
}

// K and silu as template arguments.
#define SEQCONV_CASES(CALL)                                                                            \
    switch (K) {                                                                                       \
        case 1: if (silu) CALL(1, true); else CALL(1, false); break;                                   \
        case 2: if (silu) CALL(2, true); else CALL(2, false); break;                                   \
        case 3: if (silu) CALL(3, true); else CALL(3, false); break;                                   \
        case 4: if (silu) CALL(4, true); else CALL(4, false); break;                                   \
        case 5: if (silu) CALL(5, true); else CALL(5, false); break;                                   \
        case 6: if (silu) CALL(6, true); else CALL(6, false); break;                                   \
        case 7: if (silu) CALL(7, true); else CALL(7, false); break;                                   \
        default: if (silu) CALL(8, true); else CALL(8, false); break;                                  \
    }

template <typename T, int VEC>
void fwd_k(const Seq &s, int K, int silu, const T *x, int64_t ldx, const T *w, const float *bias, const T *state, T *y,
           int64_t ldy, T *so, hipStream_t st) {
#define CALL(KK, S) fwd<T, VEC, KK, S>(s, x, ldx, w, bias, state, y, ldy, so, st)
    SEQCONV_CASES(CALL)
#undef CALL
}

template <typename T, int VEC>
hipError_t bwd_k(const Seq &s, int K, int silu, const T *x, int64_t ldx, const T *w, const float *bias, const T *state,
           const T *dy, int64_t lddy, T *dx, int64_t lddx, float *dw, float *db, T *ds, float *part, hipStream_t st) {
#define CALL(KK, S) return bwd<T, VEC, KK, S>(s, x, ldx, w, bias, state, dy, lddy, dx, lddx, dw, db, ds, part, st)
    SEQCONV_CASES(CALL)
#undef CALL
}

template <typename T, int VEC>
void step_k(const Seq &s, int K, int silu, const T *x, int64_t ldx, const T *w, const float *bias, T *state, T *y,
            int64_t ldy, hipStream_t st) {
#define CALL(KK, S) step<T, VEC, KK, S>(s, x, ldx, w, bias, state, y, ldy, st)
    SEQCONV_CASES(CALL)
#undef CALL
}

// Channels per thread: 16 bytes of them in the forward pass, four in the backward one, whose window of
// rows, weights and sums would not fit the registers twice over.
constexpr int kBwdVec = 4;

}  // namespace

int64_t causal_bwd_workspace_floats(const Seq &s, int K) {
    return tiling(s, s.C >= kBwdVec ? kBwdVec : 1, kBwdLeast).n * (K + 1) * s.C;
}

hipError_t launch_causal_fwd(const Seq &s, bool bf16, int K, int silu, const void *x, int64_t ldx, const void *w,
                             const float *bias, const void *state, void *y, int64_t ldy, void *so, hipStream_t st) {
    const auto run = [&](auto tag, auto f) {
        typedef decltype(tag) T;
        f(s, K, silu, (const T *)x, ldx, (const T *)w, bias, (const T *)state, (T *)y, ldy, (T *)so, st);
    };
    if (bf16)
        run(uint16_t{}, s.C >= 8 ? fwd_k<uint16_t, 8> : fwd_k<uint16_t, 1>);
    else
        run(float{}, s.C >= 4 ? fwd_k<float, 4> : fwd_k<float, 1>);
    return hipGetLastError();
}

hipError_t launch_causal_bwd(const Seq &s, bool bf16, int K, int silu, const void *x, int64_t ldx, const void *w,
                             const float *bias, const void *state, const void *dy, int64_t lddy, void *dx, int64_t lddx,
                             float *dw, float *db, void *ds, float *part, hipStream_t st) {
    const auto run = [&](auto tag, auto f) {
        typedef decltype(tag) T;
        return f(s, K, silu, (const T *)x, ldx, (const T *)w, bias, (const T *)state, (const T *)dy, lddy, (T *)dx, lddx, dw, db,
          (T *)ds, part, st);
    };
    return bf16 ? run(uint16_t{}, s.C >= kBwdVec ? bwd_k<uint16_t, kBwdVec> : bwd_k<uint16_t, 1>)
                : run(float{}, s.C >= kBwdVec ? bwd_k<float, kBwdVec> : bwd_k<float, 1>);
}

hipError_t launch_causal_step(const Seq &s, bool bf16, int K, int silu, const void *x, int64_t ldx, const void *w,
                              const float *bias, void *state, void *y, int64_t ldy, hipStream_t st) {
    if (bf16)
        (s.C % 2 ? step_k<uint16_t, 1> : step_k<uint16_t, 2>)(s, K, silu, (const uint16_t *)x, ldx, (const uint16_t *)w, bias,
                                                              (uint16_t *)state, (uint16_t *)y, ldy, st);
    else
        step_k<float, 1>(s, K, silu, (const float *)x, ldx, (const float *)w, bias, (float *)state, (float *)y, ldy, st);
    return hipGetLastError();
}

}  // namespace convfwd
