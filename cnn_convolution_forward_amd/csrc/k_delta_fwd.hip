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
// The pages of K, Q, T and P (57 KB for bf16 heads of 128) are brought to LDS
// asynchronously, a block ahead where two buffers fit; values are loaded at their block's start.
//
// What bounds it: the chain itself.  A block's products depend on each other, and there is one wave to a SIMD
// (8 x 2048 tokens in 16 heads of 128: 512 waves for 1024 SIMDs, 240 us for 32 blocks of which the matrix instructions
// take 57).  Of a block's 13800 cycles K S and Q S take 3000, R with the wait for V and the operands of U 2500, U 2100, the new S
// and P U 2200, y 1800; saving the states adds 2700.  y's products in 22 bits, and powers of two for rows and for 32 tokens,
// are 30 of the 240 us.  Tried and slower, as their registers are moved to and fro: V a block ahead (323 to 337 us for the whole
// call), the states' accesses four columns wide and transposed between lanes (323 to 329).
#include "delta_common.h"

namespace convfwd {
namespace {

// SUM: without y, for what a segment makes of a state.
template <int DKB, int PARTS, bool SUM> struct FwdPages {
    static constexpr int F = 4 * DKB;                   // pages of one part of K or Q
    static constexpr int kQK = (SUM ? 1 : 2) * PARTS * F;
    // P's lo from memory, not by way of LDS, where that lets a compute unit hold two workgroups (8 x 2048 tokens in 16 heads of 64:
    // 211 us with one, 190 with two)
    static constexpr bool kLowDirect = !SUM && DKB == 2 && PARTS == 1;
    static constexpr int kTri = (SUM ? 2 : kLowDirect ? 3 : 4) * kTriPages;                 // T and P, hi and lo
    static constexpr int kAll = kQK + kTri + 1;         // and a page of the rows' factors
    static constexpr int kBuffers = 2 * kAll <= 156 ? 2 : 1;
};

template <typename T, int DKB, bool SUM>
__global__ __launch_bounds__(256) void delta_fwd_kernel(Seq s, Delta d, DeltaWs ws, int slices, const T *__restrict__ v,
                                                        int64_t ldv, const float *__restrict__ s0, T *__restrict__ y,
                                                        int64_t ldy, float *__restrict__ sT,
                                                        float *__restrict__ states) {
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 2;
    typedef FwdPages<DKB, PARTS, SUM> P;
    extern __shared__ __align__(1024) char lds[];
    const int lane = threadIdx.x & 63, half = lane >> 5, col = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    float *table = reinterpret_cast<float *>(lds + P::kBuffers * P::kAll * 1024) + wave * 96;      // three factors for each column
    const int heads = s.B * d.Hv, bh = (int)(blockIdx.x % heads);
    const int runs = SUM ? ws.segments - 1 : ws.segments, seg = (int)(blockIdx.x / heads) % runs;
    const int slice = (int)(blockIdx.x / heads) / runs * waves + wave;
    const int b = bh / d.Hv, hv = bh % d.Hv, hk = hv / d.group;
    // columns past the last are zeros and not stored; SUM: behind v's 32 slices columns those of the matrix, which start as the identity
    const int c = slice * 32 + col;
    const uint32_t at_s = c < d.Dv ? 4 * c : kOob, at_v = c < d.Dv ? (uint32_t)sizeof(T) * c : kOob;
    const uint32_t ld_s = 4 * d.Dv, ld_v = (uint32_t)(ldv * sizeof(T)), ld_y = (uint32_t)(ldy * sizeof(T));
    int64_t first;
    int len;
    seq_range(s, b, first, len);
    const int all = (len + kBlock - 1) / kBlock, begin = seg * ws.seg_blocks, blocks = min(all, begin + ws.seg_blocks);
    if (seg > 0 && begin >= all) return;                               // an empty sequence has its first segment
    if (SUM && blocks == all) return;                                  // nothing follows the last one
    const int64_t slot0 = first_block(s, ws.per, b, first);
    const int state = d.Dk * d.Dv;
    const uint32_t lds0 = lds_address(lds);
    // in front of a later segment, the state that joining left in the place of the last one's offset
    const uint32_t ld_m = 128 * slices, at_m = 4 * c;
    const int size = 32 * DKB * 32 * (slices + DKB);
    float *sums = ws.sums + ((first_segment(s, ws, b, first) + seg) * d.Hv + hv) * size;

    acc_t S[DKB];
#pragma unroll
    for (int i = 0; i < DKB; ++i) S[i] = zeros();
    if (SUM && slice >= slices) {
#pragma unroll
        for (int i = 0; i < DKB; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) S[i][r] = 32 * i + acc_row(r, half) == c - 32 * slices ? 1.f : 0.f;
    } else if (seg == 0) {
        if (s0) load_state<DKB>(make_rsrc(s0 + (int64_t)bh * state, 4 * state), at_s, ld_s, half, S);
    } else if (!SUM) {
        load_state<DKB>(make_rsrc(sums - (int64_t)d.Hv * size, 4 * size), slice < slices ? at_m : kOob, ld_m, half, S);
    }

    const auto fetch = [&](int k) {
        const uint32_t buf = lds0 + (P::kBuffers == 2 ? (k & 1) * P::kAll * 1024 : 0);
        const int64_t slot = slot0 + k, rec = slot * d.Hv + hv;
        copy_pages<P::kQK>(ws.qk + (slot * d.H + hk) * ws.qk_pages * kPage, buf, wave, waves, lane);
        copy_pages<P::kTri>(ws.tri + rec * ws.tri_pages * kPage, buf + P::kQK * 1024, wave, waves, lane);
        if (wave == waves - 1) copy1((const uint4 *)(ws.rows + rec * kRowsFloats), buf + (P::kAll - 1) * 1024, 16 * lane);
    };
    if (begin < blocks) fetch(begin);
    wait_copies();

    for (int k = begin; k < blocks; ++k) {
        // Every wave's part of the pages is there; every wave is done with the other buffer.
        __syncthreads();
        const char *buf = lds + (P::kBuffers == 2 ? (k & 1) * P::kAll * 1024 : 0);
        const int n = min(len - k * kBlock, kBlock);
        const float *rec = ws.rows + ((slot0 + k) * d.Hv + hv) * kRowsFloats;
        const float gamma = rec[kGamma], invP[2] = {rec[64 * kRowInvP + col], rec[64 * kRowInvP + 32 + col]};
        Column<T> V;
        V.load(rows_buffer(v + (first + (int64_t)k * kBlock) * ldv + hv * d.Dv, n, ldv, d.Dv), at_v, ld_v, half);
        h8_t low[2 * kTriPages];
        if constexpr (P::kLowDirect) {
            const uint4 *src = ws.tri + (((slot0 + k) * d.Hv + hv) * ws.tri_pages + 3 * kTriPages) * kPage + lane;
#pragma unroll
            for (int u = 0; u < kTriPages; ++u) low[kTriPages + u] = __builtin_bit_cast(h8_t, src[u * kPage]);
        }
        const auto page = [&](int i) { return *reinterpret_cast<const h8_t *>(buf + i * 1024 + lane * 16); };
        const float *fac = reinterpret_cast<const float *>(buf + (P::kAll - 1) * 1024);
        const auto factors = [&](int row, int t, int a) { return *reinterpret_cast<const f4_t *>(fac + 64 * row + 32 * t + 8 * a + 4 * half); };
        if (!SUM && states)
            store_state<DKB>(make_rsrc(states + (((int64_t)b * ((s.T + kBlock - 1) / kBlock) + k) * d.Hv + hv) * state, 4 * state), at_s,
                             ld_s, half, S);

        // products with S: K S for U, and (Q S)^T for y.  Pages are read a step ahead, or in front of the phase that needs them:
        // there is one wave to a SIMD, so nothing else would hide LDS's latency
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < DKB; ++i) m = max_abs(S[i], m);
        const float sc = pow2_scale(max_halves(m)), isc = pow2_inv(sc);
        acc_t X[2] = {zeros(), zeros()}, Y[2] = {zeros(), zeros()};
        constexpr int kT = P::kQK, kP = kT + 2 * kTriPages, kQ = PARTS * P::F;
        h8_t kp[2][2 * PARTS], qp[2][2 * PARTS];
        const auto read_kq = [&](int i) {
#pragma unroll
            for (int u = 0; u < 2 * PARTS; ++u) {
                kp[i & 1][u] = page((u >> 1) * P::F + (u & 1) * 2 * DKB + i);
                if constexpr (!SUM) qp[i & 1][u] = page(kQ + (u >> 1) * P::F + (u & 1) * 2 * DKB + i);
            }
        };
        read_kq(0);
        h8_t tri[2 * kTriPages];
        f4_t ek[2][4];
#pragma unroll
        for (int i = 0; i < 2 * DKB; ++i) {
            if (i + 1 < 2 * DKB) {
                read_kq(i + 1);
            } else {
#pragma unroll
                for (int u = 0; u < 2 * kTriPages; ++u) tri[u] = page(kT + u);
#pragma unroll
                for (int u = 0; u < 8; ++u) ek[u >> 2][u & 3] = factors(kRowEK, u >> 2, u & 3);
            }
            __builtin_amdgcn_sched_barrier(0);
            const Pair f = split8(sc, [&](int j) { return S[i >> 1][8 * (i & 1) + j]; });
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                X[t] = mfma(kp[i & 1][t], f.hi, X[t]);
                if constexpr (!SUM) Y[t] = mfma(f.hi, qp[i & 1][t], Y[t]);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                X[t] = mfma(kp[i & 1][t], f.lo, X[t]);
                if constexpr (!SUM) Y[t] = mfma(f.lo, qp[i & 1][t], Y[t]);
                if constexpr (PARTS == 2) {
                    X[t] = mfma(kp[i & 1][2 + t], f.hi, X[t]);
                    if constexpr (!SUM) Y[t] = mfma(f.hi, qp[i & 1][2 + t], Y[t]);
                }
            }
        }
        // R = V - E K S.  A column of it, as of U, has a power of two for each half of the tokens: tokens 32.. then cost 0..31,
        // which do not depend on them, no bits, however large they are
        acc_t Rr[2];
        float sr[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int a = 0; a < 4; ++a) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    Rr[t][4 * a + j] = fmaf(-ek[t][a][j], X[t][4 * a + j] * isc, V.get(16 * t + 4 * a + j));
            }
            sr[t] = pow2_scale(max_halves(max_abs(Rr[t])));
        }
        if (P::kBuffers == 2 && k + 1 < blocks) fetch(k + 1);           // behind V's loads, which would wait for it
        h8_t kt[4 * PARTS], kt2[4 * PARTS];
        // rows 32 i .. + 31 of K^T, from the pages of K: 16 rows are a page's columns, four lanes of 8 bytes to a token
        const auto read_kt = [&](int i, h8_t(&to)[4 * PARTS]) {
            const char *p = buf + ((lane >> 4) & 1) * 1024 + ((lane & 1) * 32 + 4 * half + ((lane >> 2) & 3)) * 16 + ((lane >> 1) & 1) * 8;
#pragma unroll
            for (int u = 0; u < 4 * PARTS; ++u) {
                const char *q = p + ((u >> 2) * P::F + ((u >> 1) & 1) * 2 * DKB + 2 * i) * 1024 + (u & 1) * 256;
                const h4_t a = read_columns((const _Float16 *)q), b = read_columns((const _Float16 *)(q + 128));
#pragma unroll
                for (int j = 0; j < 4; ++j) to[u][j] = a[j], to[u][4 + j] = b[j];
            }
        };
        read_kt(0, kt);
        __builtin_amdgcn_sched_barrier(0);
        // U = T beta R: of tokens 0..31, of 32.. from R of 32.., and from R of 0..31
        acc_t part[3] = {zeros(), zeros(), zeros()};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Pair f = split8(sr[i >> 1], [&](int j) { return Rr[i >> 1][8 * (i & 1) + j]; });
            const auto to = [&](int t) -> acc_t & { return part[t + (t > i >> 1)]; };
#pragma unroll
            for (int t = i >> 1; t < 2; ++t) to(t) = mfma(tri[low_page(t, i)], f.hi, to(t));
#pragma unroll
            for (int t = i >> 1; t < 2; ++t) to(t) = mfma(tri[low_page(t, i)], f.lo, to(t));
#pragma unroll
            for (int t = i >> 1; t < 2; ++t) to(t) = mfma(tri[kTriPages + low_page(t, i)], f.hi, to(t));
        }
#pragma unroll
        for (int u = 0; u < (SUM ? 0 : P::kLowDirect ? kTriPages : 2 * kTriPages); ++u) low[u] = page(kP + u);      // in T's registers
        f4_t it[2][4], fk[2][4];
#pragma unroll
        for (int u = 0; u < 8; ++u) it[u >> 2][u & 3] = factors(kRowInvT, u >> 2, u & 3), fk[u >> 2][u & 3] = factors(kRowFK, u >> 2, u & 3);
        __builtin_amdgcn_sched_barrier(0);
        const float iu[2] = {pow2_inv(sr[0]), pow2_inv(sr[1])};
        acc_t U[2], W[2];
        float su[2] = {1.f, 1.f}, mw = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int a = 0; a < 4; ++a) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = 4 * a + j;
                    U[t][r] = (t ? fmaf(part[2][r], iu[0], part[1][r] * iu[1]) : part[0][r] * iu[0]) * it[t][a][j];
                    W[t][r] = U[t][r] * fk[t][a][j];
                }
            }
            if constexpr (!SUM) su[t] = pow2_scale(max_halves(max_abs(U[t])));
            mw = max_abs(W[t], mw);
        }
        const float sw = pow2_scale(max_halves(mw)), isw = pow2_inv(sw);
        // S = E_last S + (F K)^T U, and between its products (P U)^T for y
        Pair wf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) wf[i] = split8(sw, [&](int j) { return W[i >> 1][8 * (i & 1) + j]; });
        acc_t Z[3] = {zeros(), zeros(), zeros()};                       // as the parts of U
#pragma unroll
        for (int i = 0; i < DKB; ++i) {
            h8_t(&now)[4 * PARTS] = i & 1 ? kt2 : kt;
            if (i + 1 < DKB) read_kt(i + 1, i & 1 ? kt : kt2);
            __builtin_amdgcn_sched_barrier(0);
            acc_t a = zeros();
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                a = mfma(now[u], wf[u].hi, a);
                a = mfma(now[u], wf[u].lo, a);
                if constexpr (PARTS == 2) a = mfma(now[4 + u], wf[u].hi, a);
            }
            // every page of U in one of the DKB steps
#pragma unroll
            for (int q = i; q < (SUM ? 0 : 4); q += DKB) {
                const Pair f = split8(su[q >> 1], [&](int j) { return U[q >> 1][8 * (q & 1) + j]; });
#pragma unroll
                for (int t = q >> 1; t < 2; ++t) {
                    acc_t &to = Z[t + (t > q >> 1)];
                    to = mfma(f.hi, low[low_page(t, q)], to);
                    to = mfma(f.lo, low[low_page(t, q)], to);
                    to = mfma(f.hi, low[kTriPages + low_page(t, q)], to);
                }
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) S[i][r] = fmaf(a[r], isw, gamma * S[i][r]);
        }
        const float eq[2] = {fac[64 * kRowEQ + col], fac[64 * kRowEQ + 32 + col]};
        if (P::kBuffers == 1 && k + 1 < blocks) {
            __syncthreads();                                           // every wave is done with the pages
            fetch(k + 1);
        }
        wait_copies();                                                 // in front of y's stores, which take longer
        if constexpr (SUM) continue;
        // y: a lane has token 32 t + col, columns 8 a + 4 half + 0..3 of the slice.  The factors of columns come from the lanes
        // that made them, through LDS (within the wave: the hardware keeps LDS accesses of a wave in order).
        if (half == 0) table[col] = isc, table[32 + col] = pow2_inv(su[0]), table[64 + col] = pow2_inv(su[1]);
        __builtin_amdgcn_wave_barrier();
        const __amdgpu_buffer_rsrc_t ry = rows_buffer(y + (first + (int64_t)k * kBlock) * ldy + hv * d.Dv, n, ldy, d.Dv);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int row = 32 * t + col, c0 = slice * 32 + 4 * half;
            const uint32_t off = row * ld_y + c0 * (uint32_t)sizeof(T);
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const f4_t fs = *reinterpret_cast<const f4_t *>(table + 8 * a + 4 * half);
                const f4_t f0 = *reinterpret_cast<const f4_t *>(table + 32 + 8 * a + 4 * half);
                const f4_t f1 = *reinterpret_cast<const f4_t *>(table + 64 + 8 * a + 4 * half);
                float o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = 4 * a + j;
                    o[j] = fmaf(Y[t][r] * fs[j], eq[t], (t ? fmaf(Z[2][r], f0[j], Z[1][r] * f1[j]) : Z[0][r] * f0[j]) * invP[t]);
                }
                store4(ry, off + 8 * a * (uint32_t)sizeof(T), d.Dv - c0 - 8 * a, d.Dv & 3, o, y);
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
    if constexpr (SUM) {
        store_sum<DKB>(sums, slices, slice, lane, S);
        return;
    }
    if (sT && blocks == all) store_state<DKB>(make_rsrc(sT + (int64_t)bh * state, 4 * state), at_s, ld_s, half, S);
}

template <typename T, int DKB, bool SUM>
hipError_t chain(const Seq &s, const Delta &d, const DeltaWs &ws, const DeltaIn &in, const float *s0, RowsOut y, float *sT,
                 float *states, hipStream_t st) {
    typedef FwdPages<DKB, sizeof(T) == 2 ? 1 : 2, SUM> P;
    const int slices = (d.Dv + 31) / 32, columns = slices + (SUM ? DKB : 0);
    const int64_t chains = (int64_t)s.B * d.Hv * (SUM ? ws.segments - 1 : ws.segments);
    const int waves = waves_of(chains, columns);
    const int bytes = P::kBuffers * P::kAll * 1024 + waves * 384;
    const hipError_t e = hipFuncSetAttribute((const void *)delta_fwd_kernel<T, DKB, SUM>, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    delta_fwd_kernel<T, DKB, SUM><<<(unsigned)(chains * ((columns + waves - 1) / waves)), 64 * waves, bytes, st>>>(
        s, d, ws, slices, (const T *)in.v.p, in.v.ld, s0, (T *)y.p, y.ld, sT, states);
    return hipGetLastError();
}

template <typename T, int DKB>
hipError_t fwd(const Seq &s, const Delta &d, const DeltaWs &ws, const DeltaIn &in, const float *s0, RowsOut y, float *sT,
               float *states, hipStream_t st) {
    if (ws.segments > 1) {
        hipError_t e = chain<T, DKB, true>(s, d, ws, in, s0, y, sT, states, st);
        if (e != hipSuccess || (e = launch_delta_join(s, d, ws, false, st)) != hipSuccess) return e;
    }
    return chain<T, DKB, false>(s, d, ws, in, s0, y, sT, states, st);
}

template <typename T>
hipError_t run(const Seq &s, const Delta &d, const DeltaWs &ws, const DeltaIn &in, const float *s0, RowsOut y, float *sT,
               float *states, hipStream_t st) {
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
    if (ws.blocks > 0) launch_delta_prep(s, d, bf16, false, ws, in, delta_fill(s, {{y, d.Hv * d.Dv, bf16 ? 2 : 4}}), st);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    return bf16 ? run<uint16_t>(s, d, ws, in, s0, y, sT, states, st) : run<float>(s, d, ws, in, s0, y, sT, states, st);
}

}  // namespace convfwd
