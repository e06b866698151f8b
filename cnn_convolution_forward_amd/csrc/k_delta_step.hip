// k_delta_step.hip -- one token of the gated delta rule for each of B sequences
// (conv_delta_step).
//
//   e = v - a S^T k,   S = a S + beta k e^T,   y = scale S^T q = scale (a S^T q + (q.k) beta e),   a = exp(g)
//
// Nine operations for eight bytes of state: HBM is the bound, so S is read
// once, both products with it are taken from registers, and it is written once.
//
// A workgroup has 32 columns of one head's state: 8 threads of 4 columns by 32 of 4
// rows.  Four workgroups to a head of 128 keep the chip busy with few heads, and every
// batch uses the same layout, so that a sequence has the same bits in each.
// 64 sequences of 16 heads of 128 x 128: 25.3 us for 134 MB (5.3 TB/s); one sequence: 13 us, the call's own cost.
#include "seq_common.h"
#include "delta_internal.h"

namespace convfwd {
namespace {

constexpr int kThreads = 256, kCols = 32, kMaxDim = 128;

// Sum over the lanes of a wave that differ in lane / 8.
__device__ __forceinline__ float sum8(float v) {
    v += __shfl_xor(v, 8);
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Four floats of a row that ends at column n; zeros behind it.
__device__ __forceinline__ void load4(const float *p, int c, int n, float (&f)[4]) {
    if (c + 4 <= n) {
        load_f32<float, 4>(p + c, f);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = c + j < n ? p[c + j] : 0.f;
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void delta_step_kernel(Delta d, int slices, const T *__restrict__ q, int64_t ldq,
                                                              const T *__restrict__ k, int64_t ldk, const T *__restrict__ v,
                                                              int64_t ldv, const float *__restrict__ g, int64_t ldg,
                                                              const float *__restrict__ beta, int64_t ldb,
                                                              float *__restrict__ S, T *__restrict__ y, int64_t ldy) {
    __shared__ float qk[2][kMaxDim], part[4][2 * kCols + 1];
    __shared__ double size[4];
    const int slice = blockIdx.x % slices;
    const int64_t bh = blockIdx.x / slices;
    const int b = (int)(bh / d.Hv), h = (int)(bh % d.Hv), hk = h / d.group;
    const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3, wave = threadIdx.x >> 6;
    const int c = slice * kCols + 4 * tx, r0 = 4 * ty;
    float *Sp = S + bh * d.Dk * d.Dv;
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (r0 + i < d.Dk) load4(Sp + (int64_t)(r0 + i) * d.Dv, c, d.Dv, s[i]);
        else s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
    }
    const float a = expf(g[b * ldg + h]), bt = beta[b * ldb + h];
    {   // waves 0 and 1 bring the query, 2 and 3 the key
        const int which = threadIdx.x >> 7, i = threadIdx.x & 127;
        const T *p = which ? k + b * ldk : q + b * ldq;
        float f[1] = {0.f};
        if (i < d.Dk) load_f32<T, 1>(p + hk * d.Dk + i, f);
        if (d.unit) {
            double n = (double)f[0] * f[0];                             // every square is in fp64's range
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) n += __shfl_xor(n, m);
            if ((threadIdx.x & 63) == 0) size[wave] = n;
            __syncthreads();
            n = size[2 * which] + size[2 * which + 1] + (double)d.eps;
            f[0] = n == 0.0 ? 0.f : (float)(f[0] / sqrt(n));            // a row of zeros stays
        }
        qk[which][i] = f[0];
        __syncthreads();
    }
    float kf[4], at_k[4] = {}, at_q[4] = {}, dot = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float qf = qk[0][r0 + i];
        kf[i] = qk[1][r0 + i];
        dot = fmaf(qf, kf[i], dot);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[i][j] *= a;
            at_k[j] = fmaf(kf[i], s[i][j], at_k[j]);
            at_q[j] = fmaf(qf, s[i][j], at_q[j]);
        }
    }
    dot = sum8(dot);
#pragma unroll
    for (int j = 0; j < 4; ++j) at_k[j] = sum8(at_k[j]), at_q[j] = sum8(at_q[j]);
    if ((threadIdx.x & 63) < 8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) part[wave][4 * tx + j] = at_k[j], part[wave][kCols + 4 * tx + j] = at_q[j];
        if (tx == 0) part[wave][2 * kCols] = dot;
    }
    float vf[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float f[1] = {0.f};
        if (c + j < d.Dv) load_f32<T, 1>(v + b * ldv + (int64_t)h * d.Dv + c + j, f);
        vf[j] = f[0];
    }
    __syncthreads();
    const auto total = [&](int i) { return (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]); };
    dot = total(2 * kCols);
    float u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = bt * (vf[j] - total(4 * tx + j));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (r0 + i >= d.Dk) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = fmaf(kf[i], u[j], s[i][j]);
        float *p = Sp + (int64_t)(r0 + i) * d.Dv + c;
        if (c + 4 <= d.Dv) {
            store_f32(p, s[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < d.Dv) p[j] = s[i][j];
        }
    }
    if (ty == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float o[1] = {d.scale * fmaf(dot, u[j], total(kCols + 4 * tx + j))};
            if (c + j < d.Dv) store_f32(y + b * ldy + (int64_t)h * d.Dv + c + j, o);
        }
    }
}

template <typename T>
void step(const Seq &s, const Delta &d, const DeltaIn &in, float *S, RowsOut y, hipStream_t st) {
    const int slices = (d.Dv + kCols - 1) / kCols;
    delta_step_kernel<T><<<(unsigned)((int64_t)s.B * d.Hv * slices), kThreads, 0, st>>>(
        d, slices, (const T *)in.q.p, in.q.ld, (const T *)in.k.p, in.k.ld, (const T *)in.v.p, in.v.ld, (const float *)in.g.p, in.g.ld,
        (const float *)in.beta.p, in.beta.ld, S, (T *)y.p, y.ld);
}

}  // namespace

hipError_t launch_delta_step(const Seq &s, const Delta &d, bool bf16, const DeltaIn &in, float *S, RowsOut y, hipStream_t st) {
    if (bf16) step<uint16_t>(s, d, in, S, y, st);
    else step<float>(s, d, in, S, y, st);
    return hipGetLastError();
}

}  // namespace convfwd
