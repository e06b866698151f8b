// k_delta_fwd.hip -- the gated delta rule over whole sequences (conv_delta_fwd):
// block after block of 64 tokens, with T, P and the operands of k_delta_prep.hip.
//
//   U = T beta (V - E K S),   Y = scale E Q S + P U,   S = E_last S + (F K)^T U
//
// A wave owns 32 columns of one head's state, dim_k x 32 in fp32 registers, for the
// whole sequence: columns do not meet, so waves share the operands but never wait
// for each other's results.  S, R = beta (V - E K S) and U are each the result of one
// product and, converted in registers, the operand of the next (delta_common.h).
// With the operands swapped, products with S and U give Y transposed: a lane then
// has four neighbouring values of a token and stores them together.
//
// The pages of K, K^T, Q, T and P (66 KB for bf16 heads of 128) are brought to LDS
// asynchronously, a block ahead where two buffers fit.  Values are
// loaded a block ahead into registers.
#include "delta_common.h"

namespace convfwd {
namespace {

typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void global_void;

// Copies `pages` pages from global memory to LDS, the workgroup's waves in turn.
__device__ __forceinline__ void copy_pages(const uint4 *src, char *dst, int pages, int wave, int waves, int lane) {
    for (int i = wave; i < pages; i += waves)
        __builtin_amdgcn_global_load_lds((global_void *)(src + i * kPage + lane), (lds_void *)(dst + i * 1024), 16, 0, 0);
}

template <int DKB, int PARTS> struct FwdPages {
    static constexpr int F = 4 * DKB;                   // pages of one part of K, KT or Q
    static constexpr int kQK = 3 * PARTS * F;
    static constexpr int kTri = 2 * kTriPages + PARTS * kTriPages;      // T hi and lo; of P, lo only where y has 24 bits
    static constexpr int kAll = kQK + kTri + 1;         // and a page of the rows' factors
    static constexpr int kBuffers = 2 * kAll <= 156 ? 2 : 1;
};

template <typename T, int DKB>
__global__ __launch_bounds__(256) void delta_fwd_kernel(Seq s, Delta d, DeltaWs ws, int slices, const T *__restrict__ v,
                                                        int64_t ldv, const float *__restrict__ s0, T *__restrict__ y,
                                                        int64_t ldy, float *__restrict__ sT, float *__restrict__ states) {
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 2;
    typedef FwdPages<DKB, PARTS> P;
    extern __shared__ __align__(1024) char lds[];
    const int lane = threadIdx.x & 63, half = lane >> 5, col = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    float *table = reinterpret_cast<float *>(lds + P::kBuffers * P::kAll * 1024) + wave * 64;      // two factors for each column
    const int64_t bh = blockIdx.x % ((int64_t)s.B * d.Hv);
    const int slice = (int)(blockIdx.x / ((int64_t)s.B * d.Hv)) * waves + wave;
    const int b = (int)(bh / d.Hv), hv = (int)(bh % d.Hv), hk = hv / d.group;
    const int c = slice * 32 + col, cc = min(c, d.Dv - 1);             // columns past the last are computed and not stored
    const bool on = slice < slices && c < d.Dv;
    int64_t first;
    int len;
    seq_range(s, b, first, len);
    const int blocks = (len + kBlock - 1) / kBlock;
    const int64_t slot0 = first_block(s, ws.per, b, first);
    const int64_t state_at = bh * d.Dk * d.Dv;

    acc_t S[DKB];
#pragma unroll
    for (int i = 0; i < DKB; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int row = 32 * i + acc_row(r, half);
            S[i][r] = s0 && row < d.Dk ? s0[state_at + (int64_t)row * d.Dv + cc] : 0.f;
        }

    T next[32];
    float ngamma = 0.f, ninvT = 0.f, ninvP = 0.f;
    const auto fetch = [&](int k) {
        char *buf = lds + (P::kBuffers == 2 ? (k & 1) * P::kAll * 1024 : 0);
        const int64_t slot = slot0 + k, rec = slot * d.Hv + hv;
        const float *rows = ws.rows + rec * kRowsFloats;
        copy_pages(ws.qk + (slot * d.H + hk) * ws.qk_pages * kPage, buf, P::kQK, wave, waves, lane);
        copy_pages(ws.tri + rec * ws.tri_pages * kPage, buf + P::kQK * 1024, P::kTri, wave, waves, lane);
        copy_pages(reinterpret_cast<const uint4 *>(rows), buf + (P::kAll - 1) * 1024, 1, wave, waves, lane);
        ngamma = rows[kGamma], ninvT = rows[kInvT], ninvP = rows[kInvP];
        const int n = min(len - k * kBlock, kBlock);
        const T *p = v + (first + (int64_t)k * kBlock) * ldv + hv * d.Dv + cc;
#pragma unroll
        for (int i = 0; i < 32; ++i) next[i] = p[min(32 * (i >> 4) + acc_row(i & 15, half), n - 1) * ldv];
    };
    if (P::kBuffers == 2 && blocks > 0) fetch(0);

    for (int k = 0; k < blocks; ++k) {
        if (P::kBuffers == 1) {
            __syncthreads();                                           // every wave is done with the last block's pages
            fetch(k);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        const char *buf = lds + (P::kBuffers == 2 ? (k & 1) * P::kAll * 1024 : 0);
        const float gamma = ngamma, invT = ninvT, invP = ninvP;
        const int n = min(len - k * kBlock, kBlock);
        float vf[2][16];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            float f[1];
            to_f32(next[i], f);
            vf[i >> 4][i & 15] = 32 * (i >> 4) + acc_row(i & 15, half) < n ? f[0] : 0.f;
        }
        if (P::kBuffers == 2 && k + 1 < blocks) fetch(k + 1);
        const auto page = [&](int i) { return *reinterpret_cast<const h8_t *>(buf + i * 1024 + lane * 16); };
        const float *fac = reinterpret_cast<const float *>(buf + (P::kAll - 1) * 1024);
        if (states && on) {
            float *p = states + (((int64_t)b * ((s.T + kBlock - 1) / kBlock) + k) * d.Hv + hv) * d.Dk * d.Dv + c;
#pragma unroll
            for (int i = 0; i < DKB; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (32 * i + acc_row(r, half) < d.Dk) p[(32 * i + acc_row(r, half)) * d.Dv] = S[i][r];
        }

        // products with S: K S for U, and (Q S)^T for y
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < DKB; ++i) m = max_abs(S[i], m);
        const float sc = pow2_scale(max_halves(m)), isc = pow2_inv(sc);
        acc_t X[2] = {zeros(), zeros()}, Y[2] = {zeros(), zeros()};
#pragma unroll
        for (int i = 0; i < 2 * DKB; ++i) {
            const Pair f = split8([&](int j) { return S[i >> 1][8 * (i & 1) + j] * sc; });
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const h8_t kp = page(t * 2 * DKB + i), qp = page(2 * PARTS * P::F + t * 2 * DKB + i);
                X[t] = mfma(kp, f.hi, X[t]);
                X[t] = mfma(kp, f.lo, X[t]);
                Y[t] = mfma(f.hi, qp, Y[t]);
                if constexpr (PARTS == 2) {
                    X[t] = mfma(page(P::F + t * 2 * DKB + i), f.hi, X[t]);
                    Y[t] = mfma(f.lo, qp, Y[t]);
                    Y[t] = mfma(f.hi, page((2 * PARTS + 1) * P::F + t * 2 * DKB + i), Y[t]);
                }
            }
        }
        // R = beta (V - E K S)
        acc_t R[2];
        m = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const f4_t bek = *reinterpret_cast<const f4_t *>(fac + 64 * kRowBEK + 32 * t + 8 * a + 4 * half);
                const f4_t bt = *reinterpret_cast<const f4_t *>(fac + 64 * kRowBeta + 32 * t + 8 * a + 4 * half);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    R[t][4 * a + j] = bt[j] * vf[t][4 * a + j] - bek[j] * (X[t][4 * a + j] * isc);
            }
            m = max_abs(R[t], m);
        }
        const float sr = pow2_scale(max_halves(m));
        // U = T R
        constexpr int kT = P::kQK, kP = kT + 2 * kTriPages;
        acc_t U[2] = {zeros(), zeros()};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Pair f = split8([&](int j) { return R[i >> 1][8 * (i & 1) + j] * sr; });
#pragma unroll
            for (int t = i >> 1; t < 2; ++t) {
                const h8_t hi = page(kT + low_page(t, i)), lo = page(kT + kTriPages + low_page(t, i));
                U[t] = mfma(hi, f.hi, U[t]);
                U[t] = mfma(hi, f.lo, U[t]);
                U[t] = mfma(lo, f.hi, U[t]);
            }
        }
        const float iu = pow2_inv(sr) * invT;
        acc_t W[2];
        m = 0.f;
        float mw = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const f4_t fk = *reinterpret_cast<const f4_t *>(fac + 64 * kRowFK + 32 * t + 8 * a + 4 * half);
#pragma unroll
                for (int j = 0; j < 4; ++j) U[t][4 * a + j] *= iu, W[t][4 * a + j] = U[t][4 * a + j] * fk[j];
            }
            m = max_abs(U[t], m);
            mw = max_abs(W[t], mw);
        }
        // (P U)^T for y
        const float su = pow2_scale(max_halves(m)), sw = pow2_scale(max_halves(mw)), isw = pow2_inv(sw);
        acc_t Z[2] = {zeros(), zeros()};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Pair f = split8([&](int j) { return U[i >> 1][8 * (i & 1) + j] * su; });
#pragma unroll
            for (int t = i >> 1; t < 2; ++t) {
                const h8_t hi = page(kP + low_page(t, i));
                Z[t] = mfma(f.hi, hi, Z[t]);
                if constexpr (PARTS == 2) {
                    Z[t] = mfma(f.lo, hi, Z[t]);
                    Z[t] = mfma(f.hi, page(kP + kTriPages + low_page(t, i)), Z[t]);
                }
            }
        }
        // S = E_last S + (F K)^T U
        Pair wf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) wf[i] = split8([&](int j) { return W[i >> 1][8 * (i & 1) + j] * sw; });
#pragma unroll
        for (int i = 0; i < DKB; ++i) {
            acc_t a = zeros();
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const h8_t kt = page(PARTS * P::F + 4 * i + u);
                a = mfma(kt, wf[u].hi, a);
                a = mfma(kt, wf[u].lo, a);
                if constexpr (PARTS == 2) a = mfma(page((PARTS + 1) * P::F + 4 * i + u), wf[u].hi, a);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) S[i][r] = fmaf(a[r], isw, gamma * S[i][r]);
        }
        // y: a lane has token 32 t + col, columns 8 a + 4 half + 0..3 of the slice.  The factors of columns come from the lanes
        // that made them, through LDS (within the wave: the hardware keeps LDS accesses of a wave in order).
        if (half == 0) table[col] = isc, table[32 + col] = pow2_inv(su) * invP;
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int row = 32 * t + col;
            const float eq = fac[64 * kRowEQ + row];
            T *p = y + (first + (int64_t)k * kBlock + row) * ldy + hv * d.Dv + slice * 32;
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const f4_t fs = *reinterpret_cast<const f4_t *>(table + 8 * a + 4 * half);
                const f4_t fu = *reinterpret_cast<const f4_t *>(table + 32 + 8 * a + 4 * half);
                const int c0 = 8 * a + 4 * half, left = d.Dv - slice * 32 - c0;
                float o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = Y[t][4 * a + j] * fs[j] * eq + Z[t][4 * a + j] * fu[j];
                if (row < n && slice < slices) {
                    if (left >= 4) {
                        store_f32(p + c0, o);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float e[1] = {o[j]};
                            if (j < left) store_f32(p + c0 + j, e);
                        }
                    }
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
    if (sT && on) {
#pragma unroll
        for (int i = 0; i < DKB; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = 32 * i + acc_row(r, half);
                if (row < d.Dk) sT[state_at + (int64_t)row * d.Dv + c] = S[i][r];
            }
    }
}

// Rows of y that no sequence holds.
template <typename T> __global__ __launch_bounds__(256) void delta_fill_kernel(Seq s, Fill f) { fill_rows(s, f, blockIdx.x, gridDim.x); }

template <typename T, int DKB>
hipError_t fwd(const Seq &s, const Delta &d, const DeltaWs &ws, const DeltaIn &in, const float *s0, RowsOut y, float *sT,
               float *states, hipStream_t st) {
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 2;
    typedef FwdPages<DKB, PARTS> P;
    const int slices = (d.Dv + 31) / 32;
    const int64_t heads = (int64_t)s.B * d.Hv;
    // Waves of a workgroup share the pages in LDS; fewer to a workgroup where that leaves compute units empty.
    int waves = slices;
    while (waves > 1 && heads * ((slices + waves - 1) / waves) < 256) waves = (waves + 1) / 2;
    const int bytes = P::kBuffers * P::kAll * 1024 + waves * 256;
    const hipError_t e = hipFuncSetAttribute((const void *)delta_fwd_kernel<T, DKB>, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    delta_fwd_kernel<T, DKB><<<(unsigned)(heads * ((slices + waves - 1) / waves)), 64 * waves, bytes, st>>>(
        s, d, ws, slices, (const T *)in.v.p, in.v.ld, s0, (T *)y.p, y.ld, sT, states);
    return hipGetLastError();
}

template <typename T>
hipError_t run(const Seq &s, const Delta &d, const DeltaWs &ws, const DeltaIn &in, const float *s0, RowsOut y, float *sT,
               float *states, hipStream_t st) {
    const Fill f = fill_of<T>(s, 4, {(T *)y.p}, {y.ld});
    if (f.blocks) delta_fill_kernel<T><<<f.blocks, 256, 0, st>>>(s, f);
    switch ((d.Dk + 31) / 32) {
    case 1: return fwd<T, 1>(s, d, ws, in, s0, y, sT, states, st);
    case 2: return fwd<T, 2>(s, d, ws, in, s0, y, sT, states, st);
    case 3: return fwd<T, 3>(s, d, ws, in, s0, y, sT, states, st);
    default: return fwd<T, 4>(s, d, ws, in, s0, y, sT, states, st);
    }
}

}  // namespace

size_t delta_fwd_workspace(const Seq &s, const Delta &d, bool bf16) {
    DeltaWs ws;
    return (size_t)delta_layout(s, d, bf16, false, nullptr, ws);
}

hipError_t launch_delta_fwd(const Seq &s, const Delta &d, bool bf16, const DeltaIn &in, const float *s0, RowsOut y, float *sT,
                            float *states, void *base, hipStream_t st) {
    DeltaWs ws;
    delta_layout(s, d, bf16, false, base, ws);
    if (ws.blocks > 0) launch_delta_prep(s, d, bf16, false, ws, in, st);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return bf16 ? run<uint16_t>(s, d, ws, in, s0, y, sT, states, st) : run<float>(s, d, ws, in, s0, y, sT, states, st);
}

}  // namespace convfwd
