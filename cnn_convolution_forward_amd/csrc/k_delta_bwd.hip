// k_delta_bwd.hip -- gradients of the gated delta rule (conv_delta_bwd), in blocks
// of 64 tokens with the operands of k_delta_prep.hip.  With dS the gradient of the
// state behind a block, and R = beta (V - E K S), U = T R as in the forward pass:
//
//   Z  = T^T (P^T dY + F K dS)                  gradient of R
//   dS = E_last dS + (scale E Q)^T dY - (beta E K)^T Z          in front of the block
//   B  = scale D (dY U^T),   M = -D (Z U^T) strictly below the diagonal
//   dq = scale E dY S^T + B K
//   dk = beta read + write,   read = M K - E Z S^T,   write = B^T Q + (beta M)^T K + F U dS^T
//   dv = beta Z,   dbeta = Z.v + k.read
//   dg = sum over the block's later tokens of (q.dq + beta k.read - k.write) + <S', dS>,
//   <S', dS> = E_last <S, dS> + sum_j k_j.(F U dS^T)_j           S' the state behind the block
//
// dg: a token's products with what was written before it grow with G, what it
// writes itself shrinks with it, so the gradients of queries and keys hold all terms.
//
// The chain over blocks needs only dS, so two kernels: the first walks through the
// blocks backwards with dS in registers, exactly like the forward pass, and leaves dS
// behind every block in the workspace; the second takes all blocks at once, with
// the saved S in front and dS behind each.
#include <type_traits>

#include "delta_common.h"

namespace convfwd {
namespace {

// ---- the chain ----

template <int DKB, int PARTS> struct ChainPages {
    static constexpr int F = 4 * DKB;
    static constexpr int kK = 2 * PARTS * F, kQT = PARTS * F;           // K and KT; QT
    static constexpr int kTri = 4 * kTriPages;                          // TT, PT, hi and lo
    static constexpr int kAll = kK + kQT + kTri + 1;
    static constexpr int kBuffers = 2 * kAll <= 156 ? 2 : 1;
};

template <typename T, int DKB>
__global__ __launch_bounds__(256) void delta_chain_kernel(Seq s, Delta d, DeltaWs ws, int slices, const T *__restrict__ dy,
                                                          int64_t lddy, const float *__restrict__ dsT, float *__restrict__ ds0) {
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 2;
    typedef ChainPages<DKB, PARTS> P;
    extern __shared__ __align__(1024) char lds[];
    const int lane = threadIdx.x & 63, half = lane >> 5, col = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int heads = s.B * d.Hv, bh = (int)(blockIdx.x % heads);
    const int slice = (int)(blockIdx.x / heads) * waves + wave;
    const int b = bh / d.Hv, hv = bh % d.Hv, hk = hv / d.group;
    const int c = slice * 32 + col;
    const uint32_t at_s = c < d.Dv ? 4 * c : kOob, at_v = c < d.Dv ? (uint32_t)sizeof(T) * c : kOob;
    const uint32_t ld_s = 4 * d.Dv, ld_v = (uint32_t)(lddy * sizeof(T));
    const uint32_t at_e = slice < slices ? 4 * c : kOob, ld_e = 128 * slices;
    int64_t first;
    int len;
    seq_range(s, b, first, len);
    const int blocks = (len + kBlock - 1) / kBlock;
    const int64_t slot0 = first_block(s, ws.per, b, first);
    const int state = d.Dk * d.Dv;
    const uint32_t lds0 = lds_address(lds);

    acc_t S[DKB];
#pragma unroll
    for (int i = 0; i < DKB; ++i) S[i] = zeros();
    if (dsT) load_state<DKB>(make_rsrc(dsT + (int64_t)bh * state, 4 * state), at_s, ld_s, half, S);

    const auto fetch = [&](int k) {
        const uint32_t buf = lds0 + (P::kBuffers == 2 ? (k & 1) * P::kAll * 1024 : 0);
        const int64_t slot = slot0 + k, rec = slot * d.Hv + hv;
        const uint4 *qk = ws.qk + (slot * d.H + hk) * ws.qk_pages * kPage;
        copy_pages<P::kK>(qk, buf, wave, waves, lane);
        copy_pages<P::kQT>(qk + 3 * PARTS * P::F * kPage, buf + P::kK * 1024, wave, waves, lane);
        copy_pages<P::kTri>(ws.tri + (rec * ws.tri_pages + 2 * kTriPages) * kPage, buf + (P::kK + P::kQT) * 1024, wave, waves, lane);
        if (wave == waves - 1) copy1((const uint4 *)(ws.rows + rec * kRowsFloats), buf + (P::kAll - 1) * 1024, 16 * lane);
    };
    if (blocks > 0) fetch(blocks - 1);
    wait_copies();

    for (int k = blocks - 1; k >= 0; --k) {
        __syncthreads();
        const char *buf = lds + (P::kBuffers == 2 ? (k & 1) * P::kAll * 1024 : 0);
        const int n = min(len - k * kBlock, kBlock);
        const int64_t at = (slot0 + k) * d.Hv + hv;
        const float *rec = ws.rows + at * kRowsFloats;
        const float gamma = rec[kGamma], invT = rec[kInvT], invP = rec[kInvP];
        Column<T> dY;
        dY.load(rows_buffer(dy + (first + (int64_t)k * kBlock) * lddy + hv * d.Dv, n, lddy, d.Dv), at_v, ld_v, half);
        const auto page = [&](int i) { return *reinterpret_cast<const h8_t *>(buf + i * 1024 + lane * 16); };
        const float *fac = reinterpret_cast<const float *>(buf + (P::kAll - 1) * 1024);
        const auto factors = [&](int row, int t, int a) { return *reinterpret_cast<const f4_t *>(fac + 64 * row + 32 * t + 8 * a + 4 * half); };
        store_state<DKB>(make_rsrc(ws.ends + at * DKB * slices * 1024, DKB * slices * 4096), at_e, ld_e, half, S);

        // K dS; as in the forward pass, pages are read a step ahead of their products
        constexpr int kTT = P::kK + P::kQT, kPT = kTT + 2 * kTriPages;
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < DKB; ++i) m = max_abs(S[i], m);
        const float sc = pow2_scale(max_halves(m)), isc = pow2_inv(sc);
        acc_t X[2] = {zeros(), zeros()};
        h8_t kp[2][2 * PARTS], pt[2 * kTriPages];
        const auto read_k = [&](int i) {
#pragma unroll
            for (int u = 0; u < 2 * PARTS; ++u) kp[i & 1][u] = page((u >> 1) * P::F + (u & 1) * 2 * DKB + i);
        };
        read_k(0);
#pragma unroll
        for (int i = 0; i < 2 * DKB; ++i) {
            if (i + 1 < 2 * DKB) {
                read_k(i + 1);
            } else {
#pragma unroll
                for (int u = 0; u < 2 * kTriPages; ++u) pt[u] = page(kPT + u);
            }
            __builtin_amdgcn_sched_barrier(0);
            const Pair f = split8(sc, [&](int j) { return S[i >> 1][8 * (i & 1) + j]; });
#pragma unroll
            for (int t = 0; t < 2; ++t) X[t] = mfma(kp[i & 1][t], f.hi, X[t]);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                X[t] = mfma(kp[i & 1][t], f.lo, X[t]);
                if constexpr (PARTS == 2) X[t] = mfma(kp[i & 1][2 + t], f.hi, X[t]);
            }
        }
        // P^T dY
        m = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) m = fmaxf(m, fabsf(dY.get(i)));
        const float so = pow2_scale(max_halves(m));
        if (P::kBuffers == 2 && k > 0) fetch(k - 1);
        acc_t W[2] = {zeros(), zeros()};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            Pair f;
            if constexpr (PARTS == 2) f = split8(so, [&](int j) { return dY.get(8 * i + j); });
            else f.hi = half8(so, [&](int j) { return dY.get(8 * i + j); });        // exact
#pragma unroll
            for (int t = 0; t <= i >> 1; ++t) {
                const int u = high_page(t, i);
                W[t] = mfma(pt[u], f.hi, W[t]);
                W[t] = mfma(pt[kTriPages + u], f.hi, W[t]);
                if constexpr (PARTS == 2) W[t] = mfma(pt[u], f.lo, W[t]);
            }
        }
        f4_t fk[2][4];
#pragma unroll
        for (int u = 0; u < 8; ++u) fk[u >> 2][u & 3] = factors(kRowFK, u >> 2, u & 3);
        h8_t tt[2 * kTriPages];
#pragma unroll
        for (int u = 0; u < 2 * kTriPages; ++u) tt[u] = page(kTT + u);
        // gradient of U
        const float ip = pow2_inv(so) * invP;
        m = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int j = 0; j < 4; ++j) X[t][4 * a + j] = fmaf(fk[t][a][j] * isc, X[t][4 * a + j], W[t][4 * a + j] * ip);
            m = max_abs(X[t], m);
        }
        const float sx = pow2_scale(max_halves(m));
        acc_t Z[2] = {zeros(), zeros()};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Pair f = split8(sx, [&](int j) { return X[i >> 1][8 * (i & 1) + j]; });
#pragma unroll
            for (int t = 0; t <= i >> 1; ++t) Z[t] = mfma(tt[high_page(t, i)], f.hi, Z[t]);
#pragma unroll
            for (int t = 0; t <= i >> 1; ++t) Z[t] = mfma(tt[high_page(t, i)], f.lo, Z[t]);
#pragma unroll
            for (int t = 0; t <= i >> 1; ++t) Z[t] = mfma(tt[kTriPages + high_page(t, i)], f.hi, Z[t]);
        }
        f4_t eq[2][4], ek[2][4], bt[2][4];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            eq[u >> 2][u & 3] = factors(kRowEQ, u >> 2, u & 3);
            ek[u >> 2][u & 3] = factors(kRowEK, u >> 2, u & 3);
            bt[u >> 2][u & 3] = factors(kRowBeta, u >> 2, u & 3);
        }
        // dS
        const float iz = pow2_inv(sx) * invT;
        m = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = 4 * a + j;
                    Z[t][r] = -(Z[t][r] * iz) * (ek[t][a][j] * bt[t][a][j]);
                    W[t][r] = eq[t][a][j] * dY.get(16 * t + r);
                }
            m = max_abs(W[t], max_abs(Z[t], m));
        }
        const float sw = pow2_scale(max_halves(m)), isw = pow2_inv(sw);
        Pair zf[4], wf[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            zf[i] = split8(sw, [&](int j) { return Z[i >> 1][8 * (i & 1) + j]; });
            wf[i] = split8(sw, [&](int j) { return W[i >> 1][8 * (i & 1) + j]; });
        }
        h8_t ka[2][8 * PARTS];
        const auto read_t = [&](int i) {
#pragma unroll
            for (int u = 0; u < 4 * PARTS; ++u) {
                ka[i & 1][u] = page((PARTS + (u >> 2)) * P::F + 4 * i + (u & 3));
                ka[i & 1][4 * PARTS + u] = page(P::kK + (u >> 2) * P::F + 4 * i + (u & 3));
            }
        };
        read_t(0);
#pragma unroll
        for (int i = 0; i < DKB; ++i) {
            if (i + 1 < DKB) read_t(i + 1);
            __builtin_amdgcn_sched_barrier(0);
            acc_t a = zeros(), e = zeros();
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const h8_t kt = ka[i & 1][u], qt = ka[i & 1][4 * PARTS + u];
                a = mfma(kt, zf[u].hi, a);
                e = mfma(qt, wf[u].hi, e);
                a = mfma(kt, zf[u].lo, a);
                e = mfma(qt, wf[u].lo, e);
                if constexpr (PARTS == 2) {
                    a = mfma(ka[i & 1][4 + u], zf[u].hi, a);
                    e = mfma(ka[i & 1][4 * PARTS + 4 + u], wf[u].hi, e);
                }
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) S[i][r] = fmaf(a[r] + e[r], isw, gamma * S[i][r]);
        }
        if (P::kBuffers == 1 && k > 0) {
            __syncthreads();                                           // every wave is done with the pages
            fetch(k - 1);
        }
        wait_copies();
    }
    if (ds0) store_state<DKB>(make_rsrc(ds0 + (int64_t)bh * state, 4 * state), at_s, ld_s, half, S);
}

// ---- the gradients of a block ----

// Pages in LDS: U and Z (lane = token, places = columns of v, hi and lo), dY (the same), and the 64x64 matrices B and M,
// each as lane = i, places = j and as lane = j, places = i.
template <int PARTS> struct GradPages {
    static constexpr int kU = 0, kZ = 32, kY = 64, kB1 = kY + 16 * PARTS, kB2 = kB1 + 2 * kTriPages, kM1 = kB2 + 2 * kTriPages,
                         kM2 = kM1 + 2 * kTriPages, kAll = kM2 + 2 * kTriPages;
};
// Floats behind the pages.
enum { kSizes = 0 /* 3 x 4 x 64: largest values of a token's U, Z, dY by slice */, kDots = 768 /* 5 x 4 x 64 */, kTotals = 2048 /* 2 x 64 */,
       kScales = 2176 /* 4: of B1, B2, M1, M2 */, kKept = 2180 /* 4 */, kBack = 2184 /* 3 x 64: inverse scales of U, Z, dY */,
       kSmall = 2376 };

// A token's dv or dk: four neighbouring values of a row, zeros past `left`.
template <typename T, bool WIDE> __device__ __forceinline__ f4_t load4(__amdgpu_buffer_rsrc_t r, uint32_t off, int left) {
    f4_t f;
    if constexpr (WIDE && sizeof(T) == 2) {
        typedef uint32_t u2_t __attribute__((ext_vector_type(2)));
        const u2_t v = __builtin_amdgcn_raw_buffer_load_b64(r, left > 0 ? (int)off : (int)kOob, 0, 0);
        f[0] = __uint_as_float(v[0] << 16), f[1] = __uint_as_float(v[0] & 0xffff0000u);
        f[2] = __uint_as_float(v[1] << 16), f[3] = __uint_as_float(v[1] & 0xffff0000u);
    } else if constexpr (WIDE) {
        const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(r, left > 0 ? (int)off : (int)kOob, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = __uint_as_float(v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int o = left > j ? (int)off + j * (int)sizeof(T) : (int)kOob;
            if constexpr (sizeof(T) == 2) f[j] = __uint_as_float((uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, o, 0, 0) << 16);
            else f[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, o, 0, 0));
        }
    }
    return f;
}

__device__ __forceinline__ float max_wave(float m) {
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) m = fmaxf(m, __shfl_xor(m, i));
    return m;
}

struct GradOut {
    RowsOut dq, dk, dv, dg, db;
    bool wide_k, wide_v, wide_s;
};

template <typename T, int DKB>
__global__ __launch_bounds__(256) void delta_grad_kernel(Seq s, Delta d, DeltaWs ws, int slices, const T *__restrict__ v,
                                                         int64_t ldv, const T *__restrict__ dy, int64_t lddy,
                                                         const float *__restrict__ states, GradOut out) {
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 2, F = 4 * DKB;
    typedef GradPages<PARTS> P;
    extern __shared__ __align__(1024) char lds[];
    float *small = reinterpret_cast<float *>(lds + P::kAll * 1024);
    const int64_t slot = blockIdx.x / d.H;
    const int hk = (int)(blockIdx.x % d.H);
    const int lane = threadIdx.x & 63, half = lane >> 5, col = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Block at = find_block(s, ws.per, slot);
    int64_t first;
    int len;
    seq_range(s, at.b, first, len);
    if (at.k < 0 || (int64_t)at.k * kBlock >= len) return;
    const int64_t r0 = first + (int64_t)at.k * kBlock;
    const int n = min(len - at.k * kBlock, kBlock);
    const uint4 *qk = ws.qk + (slot * d.H + hk) * ws.qk_pages * kPage + lane;
    const auto global_page = [&](int i) { return __builtin_bit_cast(h8_t, qk[i * kPage]); };      // K, KT, Q, QT, PARTS * F each
    const auto page = [&](int i) { return *reinterpret_cast<const h8_t *>(lds + i * 1024 + lane * 16); };
    const auto put = [&](int i, const h8_t &p) { *reinterpret_cast<h8_t *>(lds + i * 1024 + lane * 16) = p; };
    acc_t dq[2] = {zeros(), zeros()}, dk[2] = {zeros(), zeros()};        // summed over the value heads that share the key head
    if (threadIdx.x < 128) small[kTotals + threadIdx.x] = 0.f;

    for (int hv = hk * d.group; hv < (hk + 1) * d.group; ++hv) {
        const int64_t rec = slot * d.Hv + hv;
        const float *rows = ws.rows + rec * kRowsFloats;
        const double *G = reinterpret_cast<const double *>(rows + 64 * kRowG);
        const float gamma = rows[kGamma], invT = rows[kInvT], invP = rows[kInvP];
        const uint4 *tri = ws.tri + rec * ws.tri_pages * kPage + lane;
        const auto tri_page = [&](int i) { return __builtin_bit_cast(h8_t, tri[i * kPage]); };   // T, TT, PT: hi then lo
        const auto factors = [&](int row, int t, int a) { return *reinterpret_cast<const f4_t *>(rows + 64 * row + 32 * t + 8 * a + 4 * half); };
        const float *sp = states + (((int64_t)at.b * ((s.T + kBlock - 1) / kBlock) + at.k) * d.Hv + hv) * d.Dk * d.Dv;
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(sp, 4 * d.Dk * d.Dv),
                                     re = make_rsrc(ws.ends + rec * DKB * slices * 1024, DKB * slices * 4096),
                                     rv = rows_buffer(v + r0 * ldv + hv * d.Dv, n, ldv, d.Dv),
                                     rdy = rows_buffer(dy + r0 * lddy + hv * d.Dv, n, lddy, d.Dv);

        // ---- a wave to 32 columns of v: U and Z, transposed (lane = token 32 t + col, registers = columns) ----
        acc_t U[2] = {zeros(), zeros()}, Z[2] = {zeros(), zeros()};
        f4_t dyr[2][4];
        float zv[2] = {0.f, 0.f}, kept = 0.f;
        if (wave < slices) {
            const int c = 32 * wave + col;
            const uint32_t at_v = c < d.Dv ? (uint32_t)sizeof(T) * c : kOob;
            acc_t S[DKB], E[DKB];
            load_state<DKB>(rs, c < d.Dv ? 4 * c : kOob, 4 * d.Dv, half, S);
            load_state<DKB>(re, 4 * c, 128 * slices, half, E);
            float m = 0.f, me = 0.f;
#pragma unroll
            for (int i = 0; i < DKB; ++i) {
                m = max_abs(S[i], m);
                me = max_abs(E[i], me);
#pragma unroll
                for (int r = 0; r < 16; ++r) kept = fmaf(S[i][r], E[i][r], kept);
            }
            kept *= gamma;
            const float sc = pow2_scale(max_halves(m)), isc = pow2_inv(sc), se = pow2_scale(max_halves(me)), ise = pow2_inv(se);
            acc_t X[2] = {zeros(), zeros()}, W[2] = {zeros(), zeros()};
#pragma unroll
            for (int i = 0; i < 2 * DKB; ++i) {
                const Pair f = split8(sc, [&](int j) { return S[i >> 1][8 * (i & 1) + j]; });
                const Pair g = split8(se, [&](int j) { return E[i >> 1][8 * (i & 1) + j]; });
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const h8_t kp = global_page(t * 2 * DKB + i);
                    X[t] = mfma(kp, f.hi, X[t]);
                    W[t] = mfma(kp, g.hi, W[t]);
                    X[t] = mfma(kp, f.lo, X[t]);
                    W[t] = mfma(kp, g.lo, W[t]);
                    if constexpr (PARTS == 2) {
                        const h8_t kl = global_page(F + t * 2 * DKB + i);
                        X[t] = mfma(kl, f.hi, X[t]);
                        W[t] = mfma(kl, g.hi, W[t]);
                    }
                }
            }
            // U = T R
            Column<T> V;
            V.load(rv, at_v, (uint32_t)(ldv * sizeof(T)), half);
            m = 0.f;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const f4_t ek = factors(kRowEK, t, a), bt = factors(kRowBeta, t, a);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        X[t][4 * a + j] = bt[j] * fmaf(-(ek[j] * isc), X[t][4 * a + j], V.get(16 * t + 4 * a + j));
                }
                m = max_abs(X[t], m);
            }
            const float sr = pow2_scale(max_halves(m));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const Pair f = split8(sr, [&](int j) { return X[i >> 1][8 * (i & 1) + j]; });
#pragma unroll
                for (int t = i >> 1; t < 2; ++t) {
                    const h8_t hi = tri_page(low_page(t, i)), lo = tri_page(kTriPages + low_page(t, i));
                    U[t] = mfma(f.hi, hi, U[t]);
                    U[t] = mfma(f.lo, hi, U[t]);
                    U[t] = mfma(f.hi, lo, U[t]);
                }
            }
            // the factor of a column differs from lane to lane before, and from register to register now
            float *table = small + kDots + wave * 64;
            if (half == 0) table[col] = pow2_inv(sr) * invT;
            // Z = T^T (P^T dY + F K dS)
            V.load(rdy, at_v, (uint32_t)(lddy * sizeof(T)), half);
            m = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) m = fmaxf(m, fabsf(V.get(i)));
            const float so = pow2_scale(max_halves(m)), ip = pow2_inv(so) * invP;
            acc_t Y[2] = {zeros(), zeros()};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                Pair f;
                if constexpr (PARTS == 2) f = split8(so, [&](int j) { return V.get(8 * i + j); });
                else f.hi = half8(so, [&](int j) { return V.get(8 * i + j); });
#pragma unroll
                for (int t = 0; t <= i >> 1; ++t) {
                    const h8_t hi = tri_page(4 * kTriPages + high_page(t, i)), lo = tri_page(5 * kTriPages + high_page(t, i));
                    Y[t] = mfma(hi, f.hi, Y[t]);
                    Y[t] = mfma(lo, f.hi, Y[t]);
                    if constexpr (PARTS == 2) Y[t] = mfma(hi, f.lo, Y[t]);
                }
            }
            m = 0.f;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const f4_t fk = factors(kRowFK, t, a);
#pragma unroll
                    for (int j = 0; j < 4; ++j) W[t][4 * a + j] = fmaf(fk[j] * ise, W[t][4 * a + j], Y[t][4 * a + j] * ip);
                }
                m = max_abs(W[t], m);
            }
            const float sx = pow2_scale(max_halves(m));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const Pair f = split8(sx, [&](int j) { return W[i >> 1][8 * (i & 1) + j]; });
#pragma unroll
                for (int t = 0; t <= i >> 1; ++t) {
                    const h8_t hi = tri_page(2 * kTriPages + high_page(t, i)), lo = tri_page(3 * kTriPages + high_page(t, i));
                    Z[t] = mfma(f.hi, hi, Z[t]);
                    Z[t] = mfma(f.lo, hi, Z[t]);
                    Z[t] = mfma(f.hi, lo, Z[t]);
                }
            }
            if (half == 0) table[32 + col] = pow2_inv(sx) * invT;
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const f4_t fu = *reinterpret_cast<const f4_t *>(table + 8 * a + 4 * half);
                const f4_t fz = *reinterpret_cast<const f4_t *>(table + 32 + 8 * a + 4 * half);
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) U[t][4 * a + j] *= fu[j], Z[t][4 * a + j] *= fz[j];
            }
            // dv = beta Z, Z.v, and dY by token
            const __amdgpu_buffer_rsrc_t rdv = rows_buffer((T *)out.dv.p + r0 * out.dv.ld + hv * d.Dv, n, out.dv.ld, d.Dv);
            const auto rest = [&](auto aligned) {
                constexpr bool W4 = decltype(aligned)::value;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int row = 32 * t + col, c0 = 32 * wave + 4 * half;
                    const float bt = rows[64 * kRowBeta + row];
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        const int left = d.Dv - c0 - 8 * a;
                        const uint32_t in_row = (c0 + 8 * a) * (uint32_t)sizeof(T);
                        const f4_t vr = load4<T, W4>(rv, row * (uint32_t)(ldv * sizeof(T)) + in_row, left);
                        dyr[t][a] = load4<T, W4>(rdy, row * (uint32_t)(lddy * sizeof(T)) + in_row, left);
                        float o[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            zv[t] = fmaf(Z[t][4 * a + j], vr[j], zv[t]);
                            o[j] = bt * Z[t][4 * a + j];
                        }
                        store4<W4>(rdv, row * (uint32_t)(out.dv.ld * sizeof(T)) + in_row, left, o, (T *)nullptr);
                    }
                }
            };
            if (out.wide_v) rest(std::true_type());
            else rest(std::false_type());
        }
        // a token's largest values over all slices
        {
            float mu[2] = {}, mz[2] = {}, mo[2] = {};
            if (wave < slices) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    mu[t] = max_halves(max_abs(U[t]));
                    mz[t] = max_halves(max_abs(Z[t]));
#pragma unroll
                    for (int a = 0; a < 4; ++a)
#pragma unroll
                        for (int j = 0; j < 4; ++j) mo[t] = fmaxf(mo[t], fabsf(dyr[t][a][j]));
                    mo[t] = max_halves(mo[t]);
                    zv[t] += __shfl_xor(zv[t], 32);
                }
            }
            kept = kept + __shfl_xor(kept, 32);
#pragma unroll
            for (int i = 1; i < 32; i <<= 1) kept += __shfl_xor(kept, i);
            // the other half's lanes hold the same
            const float m0 = half ? mu[1] : mu[0], m1 = half ? mz[1] : mz[0], m2 = half ? mo[1] : mo[0];
            small[kSizes + (0 * 4 + wave) * 64 + lane] = m0;
            small[kSizes + (1 * 4 + wave) * 64 + lane] = m1;
            small[kSizes + (2 * 4 + wave) * 64 + lane] = m2;
            __syncthreads();                                            // also: every wave is done with its table
            small[kDots + (4 * 4 + wave) * 64 + lane] = half ? zv[1] : zv[0];
            if (lane == 0) small[kKept + wave] = kept;
        }
        float back[3][2];                                               // inverse scales of a token's U, Z, dY
#pragma unroll
        for (int q = 0; q < 3; ++q)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float m = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w) m = fmaxf(m, small[kSizes + (q * 4 + w) * 64 + 32 * t + col]);
                back[q][t] = pow2_scale(m);
            }
        if (wave < slices) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int p = 8 * t + 2 * wave + u;
                    const Pair a = split8(back[0][t], [&](int j) { return U[t][8 * u + j]; });
                    const Pair z = split8(back[1][t], [&](int j) { return Z[t][8 * u + j]; });
                    put(P::kU + p, a.hi), put(P::kU + 16 + p, a.lo);
                    put(P::kZ + p, z.hi), put(P::kZ + 16 + p, z.lo);
                    const Pair o = split8(back[2][t], [&](int j) { return dyr[t][2 * u + (j >> 2)][j & 3]; });
                    put(P::kY + p, o.hi);
                    if constexpr (PARTS == 2) put(P::kY + 16 + p, o.lo);
                }
        }
#pragma unroll
        for (int q = 0; q < 3; ++q)
#pragma unroll
            for (int t = 0; t < 2; ++t) back[q][t] = pow2_inv(back[q][t]);
        if (wave == 0) {
#pragma unroll
            for (int q = 0; q < 3; ++q) small[kBack + 64 * q + lane] = half ? back[q][1] : back[q][0];
        }
        __syncthreads();

        // ---- B and M: wave 0 and 1 B, 2 and 3 M; the even ones with lane = i ----
        {
            const bool is_m = wave >= 2, by_i = !(wave & 1);
            const int pa = is_m ? P::kZ : P::kY;                        // rows i: Z or dY; rows j: U
            acc_t C[3];
            float m = 0.f;
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                const int ib = q ? 1 : 0, jb = q == 2 ? 1 : 0;
                acc_t x = zeros();
                for (int u = 0; u < 2 * slices; ++u) {
                    const h8_t a = page(pa + 8 * ib + u), bh = page(P::kU + 8 * jb + u), bl = page(P::kU + 16 + 8 * jb + u);
                    h8_t al = {};
                    const bool two = is_m || PARTS == 2;
                    if (two) al = page(pa + 16 + 8 * ib + u);
                    if (by_i) {
                        x = mfma(bh, a, x);
                        x = mfma(bl, a, x);
                        if (two) x = mfma(bh, al, x);
                    } else {
                        x = mfma(a, bh, x);
                        x = mfma(a, bl, x);
                        if (two) x = mfma(al, bh, x);
                    }
                }
                // the lane's own token and its factors; the other index runs over the registers
                const int mine = 32 * (by_i ? ib : jb) + col;
                const float inv_mine = small[kBack + 64 * (by_i ? (is_m ? 1 : 2) : 0) + mine];
                const double g_mine = G[mine];
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int other = 32 * (by_i ? jb : ib) + acc_row(r, half);
                    const int i = by_i ? mine : other, j = by_i ? other : mine;
                    const bool in = is_m ? j < i : j <= i;
                    const float D = expf((float)(by_i ? g_mine - G[other] : G[other] - g_mine));
                    // what the contraction's index brings along: lane = i: keys j; lane = j: queries i, or beta and keys i
                    float f = by_i ? rows[64 * kRowKK + other] : is_m ? rows[64 * kRowBeta + other] * rows[64 * kRowKK + other] : rows[64 * kRowKQ + other];
                    f *= is_m ? -D : d.scale * D;
                    const float inv_other = small[kBack + 64 * (by_i ? 0 : is_m ? 1 : 2) + other];
                    x[r] = in ? x[r] * (inv_mine * inv_other) * f : 0.f;
                }
                C[q] = x;
                m = max_abs(x, m);
            }
            const float sc = pow2_scale(max_wave(m));
            const int to = is_m ? (by_i ? P::kM1 : P::kM2) : (by_i ? P::kB1 : P::kB2);
#pragma unroll
            for (int q = 0; q < 3; ++q)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int ib = q ? 1 : 0, jb = q == 2 ? 1 : 0;
                    const int p = to + (by_i ? low_page(ib, 2 * jb + u) : high_page(jb, 2 * ib + u));
                    const Pair f = split8(sc, [&](int j) { return C[q][8 * u + j]; });
                    put(p, f.hi);
                    put(kTriPages + p, f.lo);
                }
            if (lane == 0) small[kScales + wave] = pow2_inv(sc);
        }
        __syncthreads();

        // ---- a wave to 32 rows of the state: dq, read and write, transposed (lane = token, registers = dk) ----
        float dot[4][2] = {};
        acc_t q1[2], wr[2], rd[2];
        if (wave < DKB) {
            // products with S and dS: rows of the state are the operand's rows, under one power of two
            const int row = 32 * wave + col;
            const auto state_pages = [&](__amdgpu_buffer_rsrc_t r, bool padded, f4_t(&f)[16]) {
                const uint32_t ld = padded ? 128 * slices : 4 * d.Dv;
                const int width = padded ? 32 * slices : d.Dv;
#pragma unroll
                for (int u = 0; u < 16; ++u) {                          // columns 8 u + 4 half + 0..3
                    if (u >= 4 * slices) {
                        f[u] = f4_t{0.f, 0.f, 0.f, 0.f};
                        continue;
                    }
                    const int c0 = 8 * u + 4 * half;
                    if (padded || out.wide_s) f[u] = load4<float, true>(r, row * ld + 4 * c0, width - c0);
                    else f[u] = load4<float, false>(r, row * ld + 4 * c0, width - c0);
                }
                float m = 0.f;
#pragma unroll
                for (int u = 0; u < 16; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) m = fmaxf(m, fabsf(f[u][j]));
                return pow2_scale(max_wave(m));
            };
            f4_t f[16];
            acc_t q0[2] = {zeros(), zeros()}, r0[2] = {zeros(), zeros()}, w0[2] = {zeros(), zeros()};
            const float ss = state_pages(rs, false, f), iss = pow2_inv(ss);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (u >= 2 * slices) break;
                const Pair a = split8(ss, [&](int j) { return f[2 * u + (j >> 2)][j & 3]; });
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const h8_t o = page(P::kY + 8 * t + u), zh = page(P::kZ + 8 * t + u), zl = page(P::kZ + 16 + 8 * t + u);
                    q0[t] = mfma(a.hi, o, q0[t]);
                    r0[t] = mfma(a.hi, zh, r0[t]);
                    q0[t] = mfma(a.lo, o, q0[t]);
                    r0[t] = mfma(a.lo, zh, r0[t]);
                    if constexpr (PARTS == 2) q0[t] = mfma(a.hi, page(P::kY + 16 + 8 * t + u), q0[t]);
                    r0[t] = mfma(a.hi, zl, r0[t]);
                }
            }
            const float se = state_pages(re, true, f), ise = pow2_inv(se);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (u >= 2 * slices) break;
                const Pair a = split8(se, [&](int j) { return f[2 * u + (j >> 2)][j & 3]; });
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const h8_t uh = page(P::kU + 8 * t + u), ul = page(P::kU + 16 + 8 * t + u);
                    w0[t] = mfma(a.hi, uh, w0[t]);
                    w0[t] = mfma(a.lo, uh, w0[t]);
                    w0[t] = mfma(a.hi, ul, w0[t]);
                }
            }
            // products of keys and queries with B and M
            acc_t bq[2] = {zeros(), zeros()}, bw[2] = {zeros(), zeros()}, mr[2] = {zeros(), zeros()}, mw[2] = {zeros(), zeros()};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const h8_t kt = global_page(PARTS * F + 4 * wave + u), qt = global_page(3 * PARTS * F + 4 * wave + u);
                h8_t kl = {}, ql = {};
                if constexpr (PARTS == 2) kl = global_page((PARTS + 1) * F + 4 * wave + u), ql = global_page((3 * PARTS + 1) * F + 4 * wave + u);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (t >= u >> 1) {
                        const int p = low_page(t, u);
                        const h8_t b = page(P::kB1 + p), c = page(P::kM1 + p);
                        bq[t] = mfma(kt, b, bq[t]);
                        mr[t] = mfma(kt, c, mr[t]);
                        bq[t] = mfma(kt, page(P::kB1 + kTriPages + p), bq[t]);
                        mr[t] = mfma(kt, page(P::kM1 + kTriPages + p), mr[t]);
                        if constexpr (PARTS == 2) bq[t] = mfma(kl, b, bq[t]), mr[t] = mfma(kl, c, mr[t]);
                    }
                    if (t <= u >> 1) {
                        const int p = high_page(t, u);
                        const h8_t b = page(P::kB2 + p), c = page(P::kM2 + p);
                        bw[t] = mfma(qt, b, bw[t]);
                        mw[t] = mfma(kt, c, mw[t]);
                        bw[t] = mfma(qt, page(P::kB2 + kTriPages + p), bw[t]);
                        mw[t] = mfma(kt, page(P::kM2 + kTriPages + p), mw[t]);
                        if constexpr (PARTS == 2) bw[t] = mfma(ql, b, bw[t]), mw[t] = mfma(kl, c, mw[t]);
                    }
                }
            }
            const float i1 = small[kScales], i2 = small[kScales + 1], i3 = small[kScales + 2], i4 = small[kScales + 3];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int tok = 32 * t + col;
                const float E = rows[64 * kRowE + tok], Fd = rows[64 * kRowF + tok], bt = rows[64 * kRowBeta + tok];
                const float fq = d.scale * E * iss * small[kBack + 128 + tok], fr = -E * iss * small[kBack + 64 + tok],
                            fw = Fd * ise * small[kBack + tok], kk = rows[64 * kRowKK + tok], kq = rows[64 * kRowKQ + tok];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    // the token's key and query: pages of this block of dk lie as the registers do
                    const h8_t kh = global_page(t * 2 * DKB + 2 * wave + u), qh = global_page(2 * PARTS * F + t * 2 * DKB + 2 * wave + u);
                    h8_t kl = {}, ql = {};
                    if constexpr (PARTS == 2) kl = global_page(F + t * 2 * DKB + 2 * wave + u), ql = global_page((2 * PARTS + 1) * F + t * 2 * DKB + 2 * wave + u);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int r = 8 * u + j;
                        const float kx = ((float)kh[j] + (float)kl[j]) * kk, qx = ((float)qh[j] + (float)ql[j]) * kq;
                        const float w_state = w0[t][r] * fw;
                        q1[t][r] = fmaf(q0[t][r], fq, bq[t][r] * i1);
                        rd[t][r] = fmaf(r0[t][r], fr, mr[t][r] * i3);
                        wr[t][r] = w_state + fmaf(bw[t][r], i2, mw[t][r] * i4);
                        dot[0][t] = fmaf(qx, q1[t][r], dot[0][t]);
                        dot[1][t] = fmaf(kx, rd[t][r], dot[1][t]);
                        dot[2][t] = fmaf(kx, wr[t][r], dot[2][t]);
                        dot[3][t] = fmaf(kx, w_state, dot[3][t]);
                        dq[t][r] += q1[t][r];
                        dk[t][r] += fmaf(bt, rd[t][r], wr[t][r]);
                    }
                }
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (int t = 0; t < 2; ++t) dot[q][t] += __shfl_xor(dot[q][t], 32);
            small[kDots + (q * 4 + wave) * 64 + lane] = half ? dot[q][1] : dot[q][0];
        }
        __syncthreads();
        if (wave == 0) {
            const auto total = [&](int q) {
                const float *p = small + kDots + q * 256 + lane;
                return (p[0] + p[64]) + (p[128] + p[192]);
            };
            const float bt = rows[64 * kRowBeta + lane];
            const float t0 = total(0), t1 = total(1), t2 = total(2);
            double run = (double)t0 + (double)bt * t1 - (double)t2, w = (double)total(3);
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const double o = __shfl_down(run, m);
                if (lane + m < 64) run += o;
                w += __shfl_xor(w, m);
            }
            w += (double)((small[kKept] + small[kKept + 1]) + (small[kKept + 2] + small[kKept + 3]));
            if (lane < n) {
                ((float *)out.dg.p)[(r0 + lane) * out.dg.ld + hv] = (float)(run + w);
                ((float *)out.db.p)[(r0 + lane) * out.db.ld + hv] = total(4) + t1;
            }
            small[kTotals + lane] += t0;
            small[kTotals + 64 + lane] += fmaf(bt, t1, t2);
        }
        __syncthreads();                                                // the pages and floats are free for the next head
    }
    // through the unit length: x / |x| takes the part along x out of the gradient
    if (wave < DKB) {
        const float *rows = ws.rows + (slot * d.Hv + hk * d.group) * kRowsFloats;
        const auto finish = [&](auto aligned, const RowsOut &o, acc_t(&g)[2], int which) {
            const __amdgpu_buffer_rsrc_t r = rows_buffer((T *)o.p + r0 * o.ld + hk * d.Dk, n, o.ld, d.Dk);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int tok = 32 * t + col;
                const float size = rows[64 * (which ? kRowSizeQ : kRowSizeK) + tok], kap = rows[64 * (which ? kRowKQ : kRowKK) + tok];
                const float along = d.unit ? small[kTotals + (which ? 0 : 64) + tok] * kap : 0.f;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const h8_t hi = global_page((which ? 2 * PARTS * F : 0) + t * 2 * DKB + 2 * wave + u);
                    h8_t lo = {};
                    if constexpr (PARTS == 2) lo = global_page(((which ? 2 * PARTS : 0) + 1) * F + t * 2 * DKB + 2 * wave + u);
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        float f[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float x = (float)hi[4 * a + j] + (float)lo[4 * a + j];
                            f[j] = size * (d.unit ? fmaf(-along, x, g[t][8 * u + 4 * a + j]) : g[t][8 * u + 4 * a + j]);
                        }
                        const int c0 = 32 * wave + 16 * u + 8 * a + 4 * half;
                        store4<decltype(aligned)::value>(r, tok * (uint32_t)(o.ld * sizeof(T)) + c0 * (uint32_t)sizeof(T), d.Dk - c0, f, (T *)nullptr);
                    }
                }
            }
        };
        if (out.wide_k) finish(std::true_type(), out.dq, dq, 1), finish(std::true_type(), out.dk, dk, 0);
        else finish(std::false_type(), out.dq, dq, 1), finish(std::false_type(), out.dk, dk, 0);
    }
}

// Rows of one output that no sequence holds; `units` of two bytes to a row.
__global__ __launch_bounds__(256) void delta_fill_kernel(Seq s, Fill f) { fill_rows(s, f, blockIdx.x, gridDim.x); }
void fill(const Seq &s, const RowsOut &o, int cols, int esize, hipStream_t st) {
    if (!s.fill || s.rows == 0) return;
    Fill f = {};
    f.p[0] = (uint16_t *)o.p, f.ld[0] = o.ld * (esize / 2), f.n = 1, f.units = cols * (esize / 2);
    f.blocks = (int)std::min<int64_t>((s.rows + 255) / 256, 1024);
    delta_fill_kernel<<<f.blocks, 256, 0, st>>>(s, f);
}

template <typename T, int DKB>
hipError_t bwd(const Seq &s, const Delta &d, const DeltaWs &ws, const DeltaIn &in, const float *states, Rows dy, const float *dsT,
               const GradOut &out, float *ds0, hipStream_t st) {
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 2;
    typedef ChainPages<DKB, PARTS> P;
    const int slices = (d.Dv + 31) / 32;
    const int64_t heads = (int64_t)s.B * d.Hv;
    int waves = slices;
    while (waves > 1 && heads * ((slices + waves - 1) / waves) < 256) waves = (waves + 1) / 2;
    int bytes = P::kBuffers * P::kAll * 1024;
    hipError_t e = hipFuncSetAttribute((const void *)delta_chain_kernel<T, DKB>, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    delta_chain_kernel<T, DKB><<<(unsigned)(heads * ((slices + waves - 1) / waves)), 64 * waves, bytes, st>>>(
        s, d, ws, slices, (const T *)dy.p, dy.ld, dsT, ds0);
    if ((e = hipGetLastError()) != hipSuccess || ws.blocks == 0) return e;
    bytes = GradPages<PARTS>::kAll * 1024 + kSmall * 4;
    e = hipFuncSetAttribute((const void *)delta_grad_kernel<T, DKB>, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    delta_grad_kernel<T, DKB><<<(unsigned)(ws.blocks * d.H), 256, bytes, st>>>(s, d, ws, slices, (const T *)in.v.p, in.v.ld,
                                                                              (const T *)dy.p, dy.ld, states, out);
    return hipGetLastError();
}

}  // namespace

size_t delta_bwd_workspace(const Seq &s, const Delta &d, bool bf16) {
    DeltaWs ws;
    return (size_t)delta_layout(s, d, bf16, true, nullptr, ws);
}

hipError_t launch_delta_bwd(const Seq &s, const Delta &d, bool bf16, const DeltaIn &in, const float *states, Rows dy, const float *dsT,
                            RowsOut dq, RowsOut dk, RowsOut dv, RowsOut dg, RowsOut dbeta, float *ds0, void *base, hipStream_t st) {
    DeltaWs ws;
    delta_layout(s, d, bf16, true, base, ws);
    const int e = bf16 ? 2 : 4;
    fill(s, dq, d.H * d.Dk, e, st);
    fill(s, dk, d.H * d.Dk, e, st);
    fill(s, dv, d.Hv * d.Dv, e, st);
    fill(s, dg, d.Hv, 4, st);
    fill(s, dbeta, d.Hv, 4, st);
    if (ws.blocks > 0) launch_delta_prep(s, d, bf16, true, ws, in, st);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    GradOut out{dq, dk, dv, dg, dbeta, false, false, false};
    const auto wide = [&](const void *p, int64_t ld, int dim) { return bf16 ? wide_rows<uint16_t>(p, ld, dim) : wide_rows<float>(p, ld, dim); };
    out.wide_k = wide(dq.p, dq.ld, d.Dk) && wide(dk.p, dk.ld, d.Dk);
    out.wide_v = wide(in.v.p, in.v.ld, d.Dv) && wide(dy.p, dy.ld, d.Dv) && wide(dv.p, dv.ld, d.Dv);
    out.wide_s = d.Dv % 4 == 0 && (uintptr_t)states % 16 == 0;
#define CASE(n) \
    case n: return bf16 ? bwd<uint16_t, n>(s, d, ws, in, states, dy, dsT, out, ds0, st) : bwd<float, n>(s, d, ws, in, states, dy, dsT, out, ds0, st)
    switch ((d.Dk + 31) / 32) {
        CASE(1);
        CASE(2);
        CASE(3);
        CASE(4);
    }
#undef CASE
    return hipErrorInvalidValue;
}

}  // namespace convfwd
