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
//
// 8 x 2048 tokens in 16 heads of 128, bf16, 955 to 990 us on different cards: the operands 148, the chain 245, the gradients
// 625.  The chain is bound as the forward one is.  The second kernel has one workgroup to a compute unit (its pages take
// 143 KB of LDS) and reads 1.3 GB of states and their gradients, each by columns and by rows, mostly from the caches; a block
// takes 69000 cycles, of which 4000 to 6000 wait for the states' columns, 11000 make B and M (the decays' exp2 of differences in fp64,
// four for each pair of tokens) and 12000 to 14000 are the products with the states' rows and the wait for these.  Tried and slower: the third part's loads in front of the
// second (more registers than there are: 1360 us and more), the states' columns loaded four wide and transposed (946 to 965).
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

// SUM: what a segment makes of a gradient behind it, as in the forward pass.
template <typename T, int DKB, bool SUM>
__global__ __launch_bounds__(256) void delta_chain_kernel(Seq s, Delta d, DeltaWs ws, int slices, const T *__restrict__ dy,
                                                          int64_t lddy, const float *__restrict__ dsT, float *__restrict__ ds0) {
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 2;
    typedef ChainPages<DKB, PARTS> P;
    extern __shared__ __align__(1024) char lds[];
    const int lane = threadIdx.x & 63, half = lane >> 5, col = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int heads = s.B * d.Hv, bh = (int)(blockIdx.x % heads);
    // segments from the last on, which only here ends where its sequence does
    const int runs = SUM ? ws.segments - 1 : ws.segments, seg = (int)(blockIdx.x / heads) % runs + (SUM ? 1 : 0);
    const int slice = (int)(blockIdx.x / heads) / runs * waves + wave;
    const int b = bh / d.Hv, hv = bh % d.Hv, hk = hv / d.group;
    const int c = slice * 32 + col;
    const uint32_t at_s = c < d.Dv ? 4 * c : kOob, at_v = c < d.Dv ? (uint32_t)sizeof(T) * c : kOob;
    const uint32_t ld_s = 4 * d.Dv, ld_v = (uint32_t)(lddy * sizeof(T));
    const uint32_t at_e = slice < slices ? 4 * c : kOob, ld_e = 128 * slices;
    int64_t first;
    int len;
    seq_range(s, b, first, len);
    const int all = (len + kBlock - 1) / kBlock, begin = seg * ws.seg_blocks, blocks = min(all, begin + ws.seg_blocks);
    if (seg > 0 && begin >= all) return;
    const int64_t slot0 = first_block(s, ws.per, b, first);
    const int state = d.Dk * d.Dv;
    const uint32_t lds0 = lds_address(lds);
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
    } else if (blocks == all) {
        if (dsT) load_state<DKB>(make_rsrc(dsT + (int64_t)bh * state, 4 * state), at_s, ld_s, half, S);
    } else if (!SUM) {
        load_state<DKB>(make_rsrc(sums + (int64_t)d.Hv * size, 4 * size), slice < slices ? at_m : kOob, ld_m, half, S);
    }

    const auto fetch = [&](int k) {
        const uint32_t buf = lds0 + (P::kBuffers == 2 ? (k & 1) * P::kAll * 1024 : 0);
        const int64_t slot = slot0 + k, rec = slot * d.Hv + hv;
        const uint4 *qk = ws.qk + (slot * d.H + hk) * ws.qk_pages * kPage;
        copy_pages<P::kK>(qk, buf, wave, waves, lane);
        copy_pages<P::kQT>(qk + 3 * PARTS * P::F * kPage, buf + P::kK * 1024, wave, waves, lane);
        copy_pages<P::kTri>(ws.tri + (rec * ws.tri_pages + 2 * kTriPages) * kPage, buf + (P::kK + P::kQT) * 1024, wave, waves, lane);
        if (wave == waves - 1) copy1((const uint4 *)(ws.rows + rec * kRowsFloats), buf + (P::kAll - 1) * 1024, 16 * lane);
    };
    if (begin < blocks) fetch(blocks - 1);
    wait_copies();

    for (int k = blocks - 1; k >= begin; --k) {
        __syncthreads();
        const char *buf = lds + (P::kBuffers == 2 ? (k & 1) * P::kAll * 1024 : 0);
        const int n = min(len - k * kBlock, kBlock);
        const int64_t at = (slot0 + k) * d.Hv + hv;
        const float *rec = ws.rows + at * kRowsFloats;
        const float gamma = rec[kGamma];
        Column<T> dY;
        dY.load(rows_buffer(dy + (first + (int64_t)k * kBlock) * lddy + hv * d.Dv, n, lddy, d.Dv), at_v, ld_v, half);
        const auto page = [&](int i) { return *reinterpret_cast<const h8_t *>(buf + i * 1024 + lane * 16); };
        const float *fac = reinterpret_cast<const float *>(buf + (P::kAll - 1) * 1024);
        const auto factors = [&](int row, int t, int a) { return *reinterpret_cast<const f4_t *>(fac + 64 * row + 32 * t + 8 * a + 4 * half); };
        if constexpr (!SUM) store_state<DKB>(make_rsrc(ws.ends + at * DKB * slices * 1024, DKB * slices * 4096), at_e, ld_e, half, S);

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
        // P^T dY: of tokens 0..31 from dY of 0..31, of 32.., and of 0..31 from dY of 32.., whose columns have a power of two for
        // each half of the tokens, as in the forward pass
        float so[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) so[t] = pow2_scale(max_halves(max_column(dY, t)));
        if (P::kBuffers == 2 && k > begin) fetch(k - 1);
        acc_t W[3] = {zeros(), zeros(), zeros()};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            Pair f;
            if constexpr (PARTS == 2) f = split8(so[i >> 1], [&](int j) { return dY.get(8 * i + j); });
            else f.hi = half8(so[i >> 1], [&](int j) { return dY.get(8 * i + j); });        // exact
#pragma unroll
            for (int t = 0; t <= i >> 1; ++t) {
                const int u = high_page(t, i);
                acc_t &to = W[t < i >> 1 ? 2 : t];
                to = mfma(pt[u], f.hi, to);
                to = mfma(pt[kTriPages + u], f.hi, to);
                if constexpr (PARTS == 2) to = mfma(pt[u], f.lo, to);
            }
        }
        f4_t fk[2][4], jp[2][4];
#pragma unroll
        for (int u = 0; u < 8; ++u) fk[u >> 2][u & 3] = factors(kRowFK, u >> 2, u & 3), jp[u >> 2][u & 3] = factors(kRowInvPT, u >> 2, u & 3);
        h8_t tt[2 * kTriPages];
#pragma unroll
        for (int u = 0; u < 2 * kTriPages; ++u) tt[u] = page(kTT + u);
        // gradient of U
        const float ip[2] = {pow2_inv(so[0]), pow2_inv(so[1])};
        float sx[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = 4 * a + j;
                    X[t][r] = fmaf(fk[t][a][j], X[t][r] * isc, (t ? W[1][r] * ip[1] : fmaf(W[2][r], ip[1], W[0][r] * ip[0])) * jp[t][a][j]);
                }
            sx[t] = pow2_scale(max_halves(max_abs(X[t])));
        }
        acc_t Z[3] = {zeros(), zeros(), zeros()};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Pair f = split8(sx[i >> 1], [&](int j) { return X[i >> 1][8 * (i & 1) + j]; });
            const auto to = [&](int t) -> acc_t & { return Z[t < i >> 1 ? 2 : t]; };
#pragma unroll
            for (int t = 0; t <= i >> 1; ++t) to(t) = mfma(tt[high_page(t, i)], f.hi, to(t));
#pragma unroll
            for (int t = 0; t <= i >> 1; ++t) to(t) = mfma(tt[high_page(t, i)], f.lo, to(t));
#pragma unroll
            for (int t = 0; t <= i >> 1; ++t) to(t) = mfma(tt[kTriPages + high_page(t, i)], f.hi, to(t));
        }
        f4_t eq[2][4], ez[2][4];
#pragma unroll
        for (int u = 0; u < 8; ++u) eq[u >> 2][u & 3] = factors(kRowEQ, u >> 2, u & 3), ez[u >> 2][u & 3] = factors(kRowEZ, u >> 2, u & 3);
        // dS
        const float iz[2] = {pow2_inv(sx[0]), pow2_inv(sx[1])};
        m = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = 4 * a + j;
                    Z[t][r] = -(t ? Z[1][r] * iz[1] : fmaf(Z[2][r], iz[1], Z[0][r] * iz[0])) * ez[t][a][j];
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
        // a step ahead where there are registers for it: fp32 heads of 128, 8 x 1024 tokens in 16 heads, 289 us with it (spills), 174 without
        constexpr bool kAhead = PARTS * DKB < 8;
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
            if (kAhead && i + 1 < DKB) read_t(i + 1);
            if (!kAhead && i) read_t(i);
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
        if (P::kBuffers == 1 && k > begin) {
            __syncthreads();                                           // every wave is done with the pages
            fetch(k - 1);
        }
        wait_copies();
    }
    if constexpr (SUM) {
        store_sum<DKB>(sums, slices, slice, lane, S);
        return;
    }
    if (ds0 && seg == 0) store_state<DKB>(make_rsrc(ds0 + (int64_t)bh * state, 4 * state), at_s, ld_s, half, S);
}

// ---- the gradients of a block ----

// Pages in LDS.  First, in the place of dY, B and M: K (lane = token), T, TT and PT.  Then U and Z (lane = token,
// places = columns of v, hi and lo), dY (the same), and the 64x64 matrices B and M, each as lane = i, places = j and as
// lane = j, places = i.
template <int PARTS> struct GradPages {
    static constexpr int kU = 0, kZ = 32, kY = 64, kB1 = kY + 16 * PARTS, kB2 = kB1 + 2 * kTriPages, kM1 = kB2 + 2 * kTriPages,
                         kM2 = kM1 + 2 * kTriPages, kAll = kM2 + 2 * kTriPages;
    static constexpr int kK = kY, kTri = kK + 16 * PARTS, kTT = kTri + 2 * kTriPages, kPT = kTT + 2 * kTriPages;
    static_assert(kPT + 2 * kTriPages <= kAll, "fits");
};
// Floats behind the pages.
enum { kSizes = 0 /* 3 x 4 x 64: largest values of a token's U, Z, dY by slice */, kDots = 768 /* 5 x 4 x 64 */, kTotals = 2048 /* 2 x 64 */,
       kBack = 2176 /* 3 x 64: inverse scales of U, Z, dY */, kScales = 2368 /* 4 x 64: of B1, B2, M1, M2 by token */,
       kKept = 2624 /* 4 */, kTop = 2628 /* 2 x 4: largest values of S and dS by slice */, kRec = 2636 /* the rows record */,
       kSmall = kRec + kRowsFloats };

struct GradOut {
    RowsOut dq, dk, dv, dg, db;
};

// Eight waves: in the first part waves 0..3 make U and waves 4..7 Z, of 32 columns of v each; in the second every wave has one of
// B and M by i or by j, for one block of tokens; in the third waves 0..3 have dq and what k reads, waves 4..7 what it writes, of 32
// rows of the state each.
template <typename T, int DKB>
__global__ __launch_bounds__(512) void delta_grad_kernel(Seq s, Delta d, DeltaWs ws, int slices, const T *__restrict__ v,
                                                         int64_t ldv, const T *__restrict__ dy, int64_t lddy,
                                                         const float *__restrict__ states, GradOut out) {
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 2, F = 4 * DKB;
    typedef GradPages<PARTS> P;
    extern __shared__ __align__(1024) char lds[];
    float *small = reinterpret_cast<float *>(lds + P::kAll * 1024), *rows = small + kRec;
    const int64_t slot = blockIdx.x / d.H;
    const int hk = (int)(blockIdx.x % d.H);
    int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w = wave & 3;
    const bool upper = wave >= 4;
    const Block at = find_block(s, ws.per, slot);
    int64_t first;
    int len;
    seq_range(s, at.b, first, len);
    if (at.k < 0 || (int64_t)at.k * kBlock >= len) return;
    const int64_t r0 = first + (int64_t)at.k * kBlock;
    const int n = min(len - at.k * kBlock, kBlock);
    const uint4 *qk = ws.qk + (slot * d.H + hk) * ws.qk_pages * kPage;
    const auto global_page = [&](int i) { return __builtin_bit_cast(h8_t, qk[i * kPage + lane]); };      // K, KT, Q, QT, PARTS * F each
    const auto page = [&](int i) { return *reinterpret_cast<const h8_t *>(lds + i * 1024 + lane * 16); };
    const auto put = [&](int i, const h8_t &p) { *reinterpret_cast<h8_t *>(lds + i * 1024 + lane * 16) = p; };
    acc_t sum[2] = {zeros(), zeros()};                                  // dq or dk over the value heads that share the key head
    if (threadIdx.x < 128) small[kTotals + threadIdx.x] = 0.f;

    for (int hv = hk * d.group; hv < (hk + 1) * d.group; ++hv) {
        const int64_t rec = slot * d.Hv + hv;
        // addresses and pages that are the same for every value head: keep the compiler from making all of them in front of
        // the loop, which takes a thousand registers
        asm volatile("" : "+s"(qk), "+v"(lane));
        const int half = lane >> 5, col = lane & 31;
        copy_pages<PARTS * F>(qk, lds_address(lds) + P::kK * 1024, wave, 8, lane);
        copy_pages<6 * kTriPages>(ws.tri + rec * ws.tri_pages * kPage, lds_address(lds) + P::kTri * 1024, wave, 8, lane);
        for (int i = threadIdx.x; i < kRowsFloats; i += 512) rows[i] = ws.rows[rec * kRowsFloats + i];
        const auto factors = [&](int row, int t, int a) { return *reinterpret_cast<const f4_t *>(rows + 64 * row + 32 * t + 8 * a + 4 * half); };
        const float *sp = states + (((int64_t)at.b * ((s.T + kBlock - 1) / kBlock) + at.k) * d.Hv + hv) * d.Dk * d.Dv;
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(sp, 4 * d.Dk * d.Dv),
                                     re = make_rsrc(ws.ends + rec * DKB * slices * 1024, DKB * slices * 4096);
        wait_copies();
        __syncthreads();
        const float gamma = rows[kGamma];

        // ---- U or Z, transposed: lane = token 32 t + col, registers = columns ----
        acc_t U[2] = {zeros(), zeros()};
        f4_t dyr[2][4];
        float mu[2] = {}, mo[2] = {}, top = 0.f;
        const auto first_part = [&](auto is_second) {
            constexpr bool second = decltype(is_second)::value;
            const int c = 32 * w + col;
            const uint32_t at_v = c < d.Dv ? (uint32_t)sizeof(T) * c : kOob;
            const T *src = second ? dy + r0 * lddy + hv * d.Dv : v + r0 * ldv + hv * d.Dv;
            const int64_t ld = second ? lddy : ldv;
            const __amdgpu_buffer_rsrc_t rc = rows_buffer(src, n, ld, d.Dv);
            acc_t X[2] = {zeros(), zeros()};
            {   // K S or K dS
                acc_t S[DKB];
                if constexpr (second) load_state<DKB>(re, 4 * c, 128 * slices, half, S);
                else load_state<DKB>(rs, c < d.Dv ? 4 * c : kOob, 4 * d.Dv, half, S);
#pragma unroll
                for (int i = 0; i < DKB; ++i) top = max_abs(S[i], top);
                top = max_halves(top);
                const float sc = pow2_scale(top), isc = pow2_inv(sc);
#pragma unroll
                for (int i = 0; i < 2 * DKB; ++i) {
                    const Pair f = split8(sc, [&](int j) { return S[i >> 1][8 * (i & 1) + j]; });
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const h8_t kp = page(P::kK + t * 2 * DKB + i);
                        X[t] = mfma(kp, f.hi, X[t]);
                        X[t] = mfma(kp, f.lo, X[t]);
                        if constexpr (PARTS == 2) X[t] = mfma(page(P::kK + F + t * 2 * DKB + i), f.hi, X[t]);
                    }
                }
                if constexpr (!second) {                                          // <S, dS>
                    float kept = 0.f;
#pragma unroll
                    for (int i = 0; i < DKB; ++i) {
                        acc_t E[1];
                        load_state<1>(re, 4 * c + i * 32 * 128 * slices, 128 * slices, half, E);
#pragma unroll
                        for (int r = 0; r < 16; ++r) kept = fmaf(S[i][r], E[0][r], kept);
                    }
#pragma unroll
                    for (int i = 1; i < 64; i <<= 1) kept += __shfl_xor(kept, i);
                    if (lane == 0) small[kKept + w] = gamma * kept;
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 16; ++r) X[t][r] *= isc;
            }
            Column<T> V;
            V.load(rc, at_v, (uint32_t)(ld * sizeof(T)), half);
            float sx[2];                                                // of X, a power of two for each half of the tokens
            if constexpr (!second) {                                              // R = beta (V - E K S)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        const f4_t ek = factors(kRowEKBack, t, a), bt = factors(kRowBeta, t, a);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            X[t][4 * a + j] = bt[j] * fmaf(-ek[j], X[t][4 * a + j], V.get(16 * t + 4 * a + j));
                    }
                    sx[t] = pow2_scale(max_halves(max_abs(X[t])));
                }
            } else {                                                    // P^T dY + F K dS
                float so[2], ip[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) so[t] = pow2_scale(max_halves(max_column(V, t))), ip[t] = pow2_inv(so[t]);
                acc_t Y[3] = {zeros(), zeros(), zeros()};               // the last: of tokens 0..31 from those of 32..
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    Pair f;
                    if constexpr (PARTS == 2) f = split8(so[i >> 1], [&](int j) { return V.get(8 * i + j); });
                    else f.hi = half8(so[i >> 1], [&](int j) { return V.get(8 * i + j); });
#pragma unroll
                    for (int t = 0; t <= i >> 1; ++t) {
                        const h8_t hi = page(P::kPT + high_page(t, i)), lo = page(P::kPT + kTriPages + high_page(t, i));
                        acc_t &to = Y[t < i >> 1 ? 2 : t];
                        to = mfma(hi, f.hi, to);
                        to = mfma(lo, f.hi, to);
                        if constexpr (PARTS == 2) to = mfma(hi, f.lo, to);
                    }
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        const f4_t fk = factors(kRowFK, t, a), jp = factors(kRowInvPT, t, a);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int r = 4 * a + j;
                            X[t][r] = fmaf(fk[j], X[t][r], (t ? Y[1][r] * ip[1] : fmaf(Y[2][r], ip[1], Y[0][r] * ip[0])) * jp[j]);
                        }
                    }
                    sx[t] = pow2_scale(max_halves(max_abs(X[t])));
                }
            }
            // times T or T^T, transposed: the factor of a column differs from lane to lane before, from register to register behind
            acc_t cross = zeros();                                      // what one half of the tokens has from the other
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const Pair f = split8(sx[i >> 1], [&](int j) { return X[i >> 1][8 * (i & 1) + j]; });
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (second ? t > i >> 1 : t < i >> 1) continue;
                    const int p = second ? P::kTT + high_page(t, i) : P::kTri + low_page(t, i);
                    const h8_t hi = page(p), lo = page(p + kTriPages);
                    acc_t &to = t == i >> 1 ? U[t] : cross;
                    to = mfma(f.hi, hi, to);
                    to = mfma(f.lo, hi, to);
                    to = mfma(f.hi, lo, to);
                }
            }
            float *table = small + kDots + wave * 64;
            if (half == 0) table[col] = pow2_inv(sx[0]), table[32 + col] = pow2_inv(sx[1]);
            const float *it = rows + 64 * (second ? kRowInvTT : kRowInvTBack) + col;        // of the lane's tokens
            const float it0 = it[0], it1 = it[32];
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const f4_t f0 = *reinterpret_cast<const f4_t *>(table + 8 * a + 4 * half), f1 = *reinterpret_cast<const f4_t *>(table + 32 + 8 * a + 4 * half);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = 4 * a + j;
                    U[0][r] = (second ? fmaf(cross[r], f1[j], U[0][r] * f0[j]) : U[0][r] * f0[j]) * it0;
                    U[1][r] = (second ? U[1][r] * f1[j] : fmaf(cross[r], f0[j], U[1][r] * f1[j])) * it1;
                }
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) mu[t] = max_halves(max_abs(U[t]));
            if constexpr (second) {                                               // dv = beta Z, Z.v, and dY by token
                const __amdgpu_buffer_rsrc_t rv = rows_buffer(v + r0 * ldv + hv * d.Dv, n, ldv, d.Dv),
                                             rdv = rows_buffer((T *)out.dv.p + r0 * out.dv.ld + hv * d.Dv, n, out.dv.ld, d.Dv);
                float zv[2] = {0.f, 0.f};
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int row = 32 * t + col, c0 = 32 * w + 4 * half;
                    const float bt = rows[64 * kRowBeta + row];
                    const uint32_t at_row = row * (uint32_t)(ldv * sizeof(T)), at_dy = row * (uint32_t)(lddy * sizeof(T));
                    f4_t vr[4];
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        const uint32_t in_row = (c0 + 8 * a) * (uint32_t)sizeof(T);
                        vr[a] = load4<T>(rv, at_row + in_row, d.Dv - c0 - 8 * a);
                        dyr[t][a] = load4<T>(rc, at_dy + in_row, d.Dv - c0 - 8 * a);
                    }
                    if ((d.Dv & 3) && (d.Dv >> 5) == w) {               // the wave has the last columns
                        const int last = (d.Dv & ~3) - 4 * half - 32 * w;          // of the half in which they lie, a multiple of 8
                        const int left = last & 7 ? 0 : d.Dv & 3;
                        const uint32_t in_row = (d.Dv & ~3) * (uint32_t)sizeof(T);
                        const f4_t v1 = load_rest<T>(rv, at_row + in_row, left), o1 = load_rest<T>(rc, at_dy + in_row, left);
#pragma unroll
                        for (int a = 0; a < 4; ++a)
#pragma unroll
                            for (int j = 0; j < 3; ++j) {
                                vr[a][j] = last == 8 * a ? v1[j] : vr[a][j];
                                dyr[t][a][j] = last == 8 * a ? o1[j] : dyr[t][a][j];
                            }
                    }
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        float o[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            zv[t] = fmaf(U[t][4 * a + j], vr[a][j], zv[t]);
                            mo[t] = fmaxf(mo[t], fabsf(dyr[t][a][j]));
                            o[j] = bt * U[t][4 * a + j];
                        }
                        store4(rdv, row * (uint32_t)(out.dv.ld * sizeof(T)) + (c0 + 8 * a) * (uint32_t)sizeof(T), d.Dv - c0 - 8 * a, d.Dv & 3, o, (T *)nullptr);
                    }
                    mo[t] = max_halves(mo[t]);
                    zv[t] += __shfl_xor(zv[t], 32);
                }
                small[kDots + (4 * 4 + w) * 64 + lane] = half ? zv[1] : zv[0];
            }
        };
        if (w < slices) {
            if (upper) first_part(std::true_type());
            else first_part(std::false_type());
        } else if (upper) {
            small[kDots + (4 * 4 + w) * 64 + lane] = 0.f;
        }
        if (!upper && w >= slices && lane == 0) small[kKept + w] = 0.f;
        // a token's largest values over all slices, and the states'
        small[kSizes + ((upper ? 1 : 0) * 4 + w) * 64 + lane] = half ? mu[1] : mu[0];
        if (upper) small[kSizes + (2 * 4 + w) * 64 + lane] = half ? mo[1] : mo[0];
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) top = fmaxf(top, __shfl_xor(top, i));
        if (lane == 0) small[kTop + wave] = top;
        __syncthreads();
        const auto token_scale = [&](int q, int tok) {
            const float *p = small + kSizes + q * 256 + tok;
            return pow2_scale(fmaxf(fmaxf(p[0], p[64]), fmaxf(p[128], p[192])));
        };
        if (w < slices) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float su = token_scale(upper ? 1 : 0, 32 * t + col), so = upper ? token_scale(2, 32 * t + col) : 0.f;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int p = (upper ? P::kZ : P::kU) + 8 * t + 2 * w + u;
                    const Pair a = split8(su, [&](int j) { return U[t][8 * u + j]; });
                    put(p, a.hi), put(p + 16, a.lo);
                    if (upper) {
                        const Pair o = split8(so, [&](int j) { return dyr[t][2 * u + (j >> 2)][j & 3]; });
                        put(P::kY + 8 * t + 2 * w + u, o.hi);
                        if constexpr (PARTS == 2) put(P::kY + 16 + 8 * t + 2 * w + u, o.lo);
                    }
                }
            }
        }
        if (wave < 3) small[kBack + 64 * wave + lane] = pow2_inv(token_scale(wave, lane));
        const float *tp = small + kTop;
        const float ss = pow2_scale(fmaxf(fmaxf(tp[0], tp[1]), fmaxf(tp[2], tp[3]))), se = pow2_scale(fmaxf(fmaxf(tp[4], tp[5]), fmaxf(tp[6], tp[7])));
        __syncthreads();

        // ---- B and M ----
        const auto second_part = [&](auto m_or_b, auto lane_is_i) {
            // by i: lane = i, a block of i has one or two blocks of j
            constexpr bool is_m = decltype(m_or_b)::value, by_i = decltype(lane_is_i)::value, two = is_m || PARTS == 2;
            const int pa = is_m ? P::kZ : P::kY;                        // rows i: Z or dY; rows j: U
            const double *G = reinterpret_cast<const double *>(rows + 64 * kRowG);
            const int blocks = upper ? 1 : 2;                           // waves 0..3: the block of tokens with two partners
            const int mine_b = by_i == upper ? 0 : 1;
            acc_t C[2];
            float m = 0.f;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (q >= blocks) break;
                const int other_b = upper ? mine_b : q;
                const int ib = by_i ? mine_b : other_b, jb = by_i ? other_b : mine_b;
                acc_t x = zeros();
                for (int u = 0; u < 2 * slices; ++u) {
                    const h8_t a = page(pa + 8 * ib + u), bh = page(P::kU + 8 * jb + u), bl = page(P::kU + 16 + 8 * jb + u);
                    h8_t al = {};
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
                const int mine = 32 * mine_b + col;
                const float inv_mine = small[kBack + 64 * (by_i ? (is_m ? 1 : 2) : 0) + mine], i0 = fminf(inv_mine, 1.f), i1 = fmaxf(inv_mine, 1.f);
                const double g_mine = G[mine];
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int other = 32 * other_b + acc_row(r, half);
                    const int i = by_i ? mine : other, j = by_i ? other : mine;
                    const bool in = is_m ? j < i : j <= i;
                    const float D = by_i ? decay_of(g_mine, G[other]) : decay_of(G[other], g_mine);
                    // what the contraction's index brings along: lane = i: keys j; lane = j: queries i, or beta and keys i
                    float f = rows[64 * (by_i || is_m ? kRowKK : kRowKQ) + other];
                    if (!by_i && is_m) f *= rows[64 * kRowBeta + other];
                    f *= is_m ? -D : d.scale * D;
                    const float inv_other = small[kBack + 64 * (by_i ? 0 : is_m ? 1 : 2) + other];
                    float value = x[r] * i0 * (inv_other * i1) * f;
                    asm("" : "+v"(value));                              // all of it, then a selection: no branch for each
                    x[r] = in ? value : 0.f;
                }
                C[q] = x;
                m = max_abs(x, m);
            }
            const float sc = pow2_scale(max_halves(m));                 // of the lane's row: a token's gradients cost others no bits
            const int to = is_m ? (by_i ? P::kM1 : P::kM2) : (by_i ? P::kB1 : P::kB2);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (q >= blocks) break;
                const int other_b = upper ? mine_b : q;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int p = to + (by_i ? low_page(mine_b, 2 * other_b + u) : high_page(mine_b, 2 * other_b + u));
                    const Pair f = split8(sc, [&](int j) { return C[q][8 * u + j]; });
                    put(p, f.hi);
                    put(kTriPages + p, f.lo);
                }
            }
            if (half == 0) small[kScales + 64 * w + 32 * mine_b + col] = pow2_inv(sc);
        };
        if (w == 0) second_part(std::false_type(), std::true_type());
        else if (w == 1) second_part(std::false_type(), std::false_type());
        else if (w == 2) second_part(std::true_type(), std::true_type());
        else second_part(std::true_type(), std::false_type());
        __syncthreads();

        // ---- dq and read, or write, transposed: lane = token, registers = dk; the state's rows are the operand's ----
        asm volatile("" : "+s"(qk));
        float dot[2][2] = {};
        acc_t A[2] = {zeros(), zeros()}, Bb[2] = {zeros(), zeros()};
        const auto third_part = [&](auto is_second) {
            constexpr bool second = decltype(is_second)::value;
            const int row = 32 * w + col;
            const uint32_t ld = second ? 128 * slices : 4 * d.Dv;
            const int width = second ? 32 * slices : d.Dv;
            const float sc = second ? se : ss;
            f4_t quads[16];                                             // columns 8 u + 4 half + 0..3; zeros past the state's
            h8_t kt[4 * PARTS], qt[4 * PARTS];
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                const int c0 = 8 * u + 4 * half;
                quads[u] = load4<float>(second ? re : rs, row * ld + 4 * c0, u < 4 * slices ? width - c0 : 0);
            }
            if (!second && (d.Dv & 3)) {                                // the last columns of S
                const int last = (d.Dv & ~3) - 4 * half;
                const f4_t f = load_rest<float>(rs, row * ld + 4 * (d.Dv & ~3), last & 7 ? 0 : d.Dv & 3);
#pragma unroll
                for (int u = 0; u < 16; ++u)
#pragma unroll
                    for (int j = 0; j < 3; ++j) quads[u][j] = last == 8 * u ? f[j] : quads[u][j];
            }
            __builtin_amdgcn_sched_barrier(0);
            const auto read_t = [&] {
#pragma unroll
                for (int u = 0; u < 4 * PARTS; ++u) {
                    kt[u] = global_page((PARTS + (u >> 2)) * F + 4 * w + (u & 3));
                    qt[u] = global_page(((second ? 3 : 1) * PARTS + (u >> 2)) * F + 4 * w + (u & 3));
                }
            };
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (u == 4) read_t();                                   // some of the state's registers are free by then
                if (u >= 2 * slices) continue;
                const Pair a = split8(sc, [&](int j) { return quads[2 * u + (j >> 2)][j & 3]; });
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if constexpr (second) {
                        const h8_t uh = page(P::kU + 8 * t + u), ul = page(P::kU + 16 + 8 * t + u);
                        A[t] = mfma(a.hi, uh, A[t]);
                        A[t] = mfma(a.lo, uh, A[t]);
                        A[t] = mfma(a.hi, ul, A[t]);
                    } else {
                        const h8_t o = page(P::kY + 8 * t + u), zh = page(P::kZ + 8 * t + u), zl = page(P::kZ + 16 + 8 * t + u);
                        A[t] = mfma(a.hi, o, A[t]);
                        Bb[t] = mfma(a.hi, zh, Bb[t]);
                        A[t] = mfma(a.lo, o, A[t]);
                        Bb[t] = mfma(a.lo, zh, Bb[t]);
                        if constexpr (PARTS == 2) A[t] = mfma(a.hi, page(P::kY + 16 + 8 * t + u), A[t]);
                        Bb[t] = mfma(a.hi, zl, Bb[t]);
                    }
                }
            }
            // products of keys and queries with B and M
            acc_t p1[2] = {zeros(), zeros()}, p2[2] = {zeros(), zeros()};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (second ? t > u >> 1 : t < u >> 1) continue;
                    const int p = second ? high_page(t, u) : low_page(t, u);
                    const int b0 = (second ? P::kB2 : P::kB1) + p, c0 = (second ? P::kM2 : P::kM1) + p;
                    const h8_t b = page(b0), c = page(c0);
                    p1[t] = mfma(qt[u], b, p1[t]);
                    p2[t] = mfma(kt[u], c, p2[t]);
                    p1[t] = mfma(qt[u], page(b0 + kTriPages), p1[t]);
                    p2[t] = mfma(kt[u], page(c0 + kTriPages), p2[t]);
                    if constexpr (PARTS == 2) p1[t] = mfma(qt[4 + u], b, p1[t]), p2[t] = mfma(kt[4 + u], c, p2[t]);
                }
            }
            const float iss = fminf(pow2_inv(sc), 1.f), ist = fmaxf(pow2_inv(sc), 1.f);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int tok = 32 * t + col;
                const float i1 = small[kScales + 64 * (second ? 1 : 0) + tok], i2 = small[kScales + 64 * (second ? 3 : 2) + tok];
                const float E = rows[64 * kRowE + tok], kk = rows[64 * kRowKK + tok], kq = rows[64 * kRowKQ + tok];
                // waves 0..3: of dY S^T and of Z S^T; waves 4..7: of U dS^T
                const float fa = ist * (second ? rows[64 * kRowF + tok] * small[kBack + tok] : d.scale * E * small[kBack + 128 + tok]);
                const float fb = -ist * (E * small[kBack + 64 + tok]);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    // the token's key and query: pages of this block of dk lie as the registers do
                    const int p = t * 2 * DKB + 2 * w + u;
                    const h8_t kh = global_page(p), qh = global_page(2 * PARTS * F + p);
                    h8_t kl = {}, ql = {};
                    if constexpr (PARTS == 2) kl = global_page(F + p), ql = global_page((2 * PARTS + 1) * F + p);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int q = 8 * u + j;
                        const float kx = ((float)kh[j] + (float)kl[j]) * kk;
                        if constexpr (second) {
                            const float state = A[t][q] * iss * fa;
                            A[t][q] = state + fmaf(p1[t][q], i1, p2[t][q] * i2);
                            dot[0][t] = fmaf(kx, A[t][q], dot[0][t]);
                            dot[1][t] = fmaf(kx, state, dot[1][t]);
                        } else {
                            const float qx = ((float)qh[j] + (float)ql[j]) * kq;
                            A[t][q] = fmaf(A[t][q] * iss, fa, p1[t][q] * i1);
                            Bb[t][q] = fmaf(Bb[t][q] * iss, fb, p2[t][q] * i2);
                            dot[0][t] = fmaf(qx, A[t][q], dot[0][t]);
                            dot[1][t] = fmaf(kx, Bb[t][q], dot[1][t]);
                        }
                        sum[t][q] += A[t][q];
                    }
                }
            }
        };
        if (w < DKB) {
            if (upper) third_part(std::true_type());
            else third_part(std::false_type());
        }
        // dots: q.dq, k.read, k.write, k.(F U dS^T)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int t = 0; t < 2; ++t) dot[q][t] += __shfl_xor(dot[q][t], 32);
            small[kDots + (((upper ? 2 : 0) + q) * 4 + w) * 64 + lane] = half ? dot[q][1] : dot[q][0];
        }
        __syncthreads();
        // beta read goes to the waves that have write, in the place of the pages
        float *pass = reinterpret_cast<float *>(lds) + w * 2048;
        if (!upper && w < DKB) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float bt = rows[64 * kRowBeta + 32 * t + col];
#pragma unroll
                for (int q = 0; q < 16; ++q) pass[(16 * t + q) * 64 + lane] = bt * Bb[t][q];
            }
        }
        if (wave == 0) {
            const auto total = [&](int q) {
                const float *p = small + kDots + q * 256 + lane;
                return (p[0] + p[64]) + (p[128] + p[192]);
            };
            const float bt = rows[64 * kRowBeta + lane];
            const float t0 = total(0), t1 = total(1), t2 = total(2);
            double run = (double)t0 + (double)bt * t1 - (double)t2, all = (double)total(3);
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const double o = __shfl_down(run, m);
                if (lane + m < 64) run += o;
                all += __shfl_xor(all, m);
            }
            all += (double)((small[kKept] + small[kKept + 1]) + (small[kKept + 2] + small[kKept + 3]));
            if (lane < n) {
                ((float *)out.dg.p)[(r0 + lane) * out.dg.ld + hv] = (float)(run + all);
                ((float *)out.db.p)[(r0 + lane) * out.db.ld + hv] = total(4) + t1;
            }
            small[kTotals + lane] += t0;
            small[kTotals + 64 + lane] += fmaf(bt, t1, t2);
        }
        __syncthreads();
        if (upper && w < DKB) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int q = 0; q < 16; ++q) sum[t][q] += pass[(16 * t + q) * 64 + lane];
        }
        __syncthreads();                                                // the pages and floats are free for the next head
    }
    // through the unit length: x / |x| takes the part along x out of the gradient
    const int half = lane >> 5, col = lane & 31;
    if (w < DKB) {
        const float *rec = ws.rows + (slot * d.Hv + hk * d.group) * kRowsFloats;
        const RowsOut o = upper ? out.dk : out.dq;
        const int base = upper ? 0 : 2 * PARTS * F;
        const __amdgpu_buffer_rsrc_t r = rows_buffer((T *)o.p + r0 * o.ld + hk * d.Dk, n, o.ld, d.Dk);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int tok = 32 * t + col;
            const float size = rec[64 * (upper ? kRowSizeK : kRowSizeQ) + tok], kap = rec[64 * (upper ? kRowKK : kRowKQ) + tok];
            const float along = d.unit ? small[kTotals + (upper ? 64 : 0) + tok] * kap : 0.f;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int p = base + t * 2 * DKB + 2 * w + u;
                const h8_t hi = global_page(p);
                h8_t lo = {};
                if constexpr (PARTS == 2) lo = global_page(p + F);
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    float f[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x = (float)hi[4 * a + j] + (float)lo[4 * a + j];
                        f[j] = size * (d.unit ? fmaf(-along, x, sum[t][8 * u + 4 * a + j]) : sum[t][8 * u + 4 * a + j]);
                    }
                    const int c0 = 32 * w + 16 * u + 8 * a + 4 * half;
                    store4(r, tok * (uint32_t)(o.ld * sizeof(T)) + c0 * (uint32_t)sizeof(T), d.Dk - c0, d.Dk & 3, f, (T *)nullptr);
                }
            }
        }
    }
}

template <typename T, int DKB, bool SUM>
hipError_t chain(const Seq &s, const Delta &d, const DeltaWs &ws, Rows dy, const float *dsT, float *ds0, hipStream_t st) {
    typedef ChainPages<DKB, sizeof(T) == 2 ? 1 : 2> P;
    const int slices = (d.Dv + 31) / 32, columns = slices + (SUM ? DKB : 0);
    const int64_t chains = (int64_t)s.B * d.Hv * (SUM ? ws.segments - 1 : ws.segments);
    const int waves = waves_of(chains, columns), bytes = P::kBuffers * P::kAll * 1024;
    const hipError_t e = hipFuncSetAttribute((const void *)delta_chain_kernel<T, DKB, SUM>, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    delta_chain_kernel<T, DKB, SUM><<<(unsigned)(chains * ((columns + waves - 1) / waves)), 64 * waves, bytes, st>>>(
        s, d, ws, slices, (const T *)dy.p, dy.ld, dsT, ds0);
    return hipGetLastError();
}

template <typename T, int DKB>
hipError_t bwd(const Seq &s, const Delta &d, const DeltaWs &ws, const DeltaIn &in, const float *states, Rows dy, const float *dsT,
               const GradOut &out, float *ds0, hipStream_t st) {
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 2;
    const int slices = (d.Dv + 31) / 32;
    hipError_t e;
    if (ws.segments > 1) {
        if ((e = chain<T, DKB, true>(s, d, ws, dy, dsT, ds0, st)) != hipSuccess) return e;
        if ((e = launch_delta_join(s, d, ws, true, st)) != hipSuccess) return e;
    }
    if ((e = chain<T, DKB, false>(s, d, ws, dy, dsT, ds0, st)) != hipSuccess || ws.blocks == 0) return e;
    const int bytes = GradPages<PARTS>::kAll * 1024 + kSmall * 4;
    e = hipFuncSetAttribute((const void *)delta_grad_kernel<T, DKB>, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    delta_grad_kernel<T, DKB><<<(unsigned)(ws.blocks * d.H), 512, bytes, st>>>(s, d, ws, slices, (const T *)in.v.p, in.v.ld,
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
    const Fill fill = delta_fill(s, {{dq, d.H * d.Dk, e}, {dk, d.H * d.Dk, e}, {dv, d.Hv * d.Dv, e}, {dg, d.Hv, 4}, {dbeta, d.Hv, 4}});
    if (ws.blocks > 0) launch_delta_prep(s, d, bf16, true, ws, in, fill, st);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const GradOut out{dq, dk, dv, dg, dbeta};
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
