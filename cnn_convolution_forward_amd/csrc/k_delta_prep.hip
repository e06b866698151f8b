// k_delta_prep.hip -- what a block of 64 tokens of the gated delta rule needs
// before any state is known, for all blocks at once:
//
//   G = cumulative log decays,  D[i][j] = exp(G[i] - G[j]),  A = beta_i D[i][j] k_i.k_j (j < i)
//   T = (I + A)^-1,  P = scale D[i][j] q_i.k_j (j <= i)
//
// and queries and keys as pages of fp16 operands, in both orientations.  Strides,
// packing, odd widths and the sequence's end are dealt with here; the kernels
// behind it see whole tiles, with zeros for tokens that are not there.
//
// A workgroup has one block and one key head, and walks through the value heads
// that share it.  q.k and k.k are matrix products (exact for bf16).  Differences of
// G are taken in fp64: their error is relative to the difference, whatever decays came
// before.  T: the four 16x16 blocks on the diagonal by substitution, a lane to a
// column, then the blocks below from the products T_ii A_ij T_jj on the fp32 matrix
// instructions: three levels instead of 64 steps.
//
// 8 x 2048 tokens in 16 heads of 128, bf16: 115 us forward, 148 backward, for 134 MB read and 240 (436) MB written; the
// floor of these bytes is 72 (110) us.  The rest is latency, of the loads (11200 of a workgroup's 46200
// cycles, backward 17100 of 62500), the scan of the gates (5200), the substitution and the levels (6400), with four workgroups to a
// compute unit to cover it.
#include <math.h>

#include <type_traits>

#include "delta_common.h"

namespace convfwd {
namespace {

constexpr int kThreads = 256;

// N = 8 DKB elements of a row from p + c on, of which those below `n` are there.
template <typename T, int N> __device__ __forceinline__ void load_part(const T *p, int c, int n, float (&f)[N]) {
    constexpr int VEC = sizeof(T) == 2 ? 8 : 4;
#pragma unroll
    for (int i = 0; i < N; i += VEC) {
        if (c + i + VEC <= n) {
            float t[VEC];
            load_f32<T, VEC>(p + c + i, t);
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[i + j] = t[j];
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float t[1] = {0.f};
                if (c + i + j < n) load_f32<T, 1>(p + c + i + j, t);
                f[i + j] = t[0];
            }
        }
    }
}

// Four workgroups to a compute unit where LDS has room for them, which takes 128 registers (and a few spilled): 8 x 2048 tokens in 16
// heads of 128 bf16 in 109 us instead of 126 with three, when that was tried.
constexpr int resident(int parts, int dkb) { return parts * dkb > 4 ? 2 : 4; }

template <typename T, int DKB, bool BWD>
__global__ __launch_bounds__(kThreads, resident(sizeof(T) / 2, DKB)) void delta_prep_kernel(Seq s, Delta d, DeltaWs ws, const T *__restrict__ q, int64_t ldq,
                                                              const T *__restrict__ k, int64_t ldk,
                                                              const float *__restrict__ g, int64_t ldg,
                                                              const float *__restrict__ beta, int64_t ldb) {
    constexpr int DKP = 32 * DKB, PARTS = sizeof(T) == 2 ? 1 : 2, LD = DKP + 8, N = 8 * DKB;
    typedef float Square[kBlock][65];
    typedef _Float16 Tiles[PARTS][kBlock][LD];
    // keys and queries; once their products are taken, A and T lie in their place
    constexpr int kTiles = 2 * sizeof(Tiles) > 2 * sizeof(Square) ? 2 * sizeof(Tiles) : 2 * sizeof(Square);
    __shared__ __align__(16) char shared[kTiles];
    Tiles *xs = reinterpret_cast<Tiles *>(shared);
    Square &A = *reinterpret_cast<Square *>(shared), &Ti = *reinterpret_cast<Square *>(shared + sizeof(Square));
    __shared__ double G[kBlock];
    __shared__ float kap[2][kBlock], size[2][kBlock], betas[2][kBlock];
    __shared__ float top_p[2][2][32], top_t[kBlock], top_tt[BWD ? 4 : 1][kBlock];       // largest values: of rows of P by wave and tile, of T and T^T
    const int64_t slot = blockIdx.x / d.H;
    const int hk = (int)(blockIdx.x % d.H);
    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, col = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Block at = find_block(s, ws.per, slot);
    int64_t first;
    int len;
    seq_range(s, at.b, first, len);
    if (at.k < 0 || (int64_t)at.k * kBlock >= len) return;
    const int64_t r0 = first + (int64_t)at.k * kBlock;
    const int n = min(len - at.k * kBlock, kBlock);

    // gates of the first value head; those of the others are loaded a head ahead
    float gv = 0.f, b = 0.f;
    const auto load_gates = [&](int hv) {
        if (wave == 0 && lane < n) gv = g[(r0 + lane) * ldg + hv], b = beta[(r0 + lane) * ldb + hv];
    };
    load_gates(hk * d.group);

    // rows as fp16 under their own power of two, and the factor that makes the row of it
    {
        const int row = tid >> 2, c = (tid & 3) * N;
        float f[2][N];
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            if (row < n) {
                load_part<T, N>((which ? q + (r0 + row) * ldq : k + (r0 + row) * ldk) + hk * d.Dk, c, d.Dk, f[which]);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) f[which][i] = 0.f;
            }
        }
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(f[which][i]));
            m = fmaxf(m, __shfl_xor(m, 1));
            m = fmaxf(m, __shfl_xor(m, 2));
            const float sc = pow2_scale(m);
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                h4_t hi, lo;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x = f[which][i + j] * sc;
                    ss = fmaf(x, x, ss);
                    hi[j] = (_Float16)x;
                    lo[j] = (_Float16)(x - (float)hi[j]);
                }
                *reinterpret_cast<h4_t *>(&xs[which][0][row][c + i]) = hi;
                if constexpr (PARTS == 2) *reinterpret_cast<h4_t *>(&xs[which][PARTS - 1][row][c + i]) = lo;
            }
            ss += __shfl_xor(ss, 1);
            ss += __shfl_xor(ss, 2);
            if ((tid & 3) == 0) {
                // unit length: x / sqrt(sum x^2 + eps) with sum x^2 = ss / sc^2.  A row of zeros stays, and its gradient has the
                // factor 1 / sqrt(eps) (none without eps); past fp32, eps is all of the sum.
                const float e2 = d.eps * sc * sc;
                const float f0 = !d.unit ? pow2_inv(sc) : isinf(e2) ? 1.f / (sqrtf(d.eps) * sc) : ss + e2 == 0.f ? 0.f : 1.f / sqrtf(ss + e2);
                kap[which][row] = f0;
                size[which][row] = f0 * sc;
            }
        }
    }
    __syncthreads();

    const auto row_page = [&](int which, int part, int rb, int m) {       // lane = token
        const _Float16 *p = &xs[which][part][32 * rb + col][16 * m + 4 * half];
        const h4_t a = *reinterpret_cast<const h4_t *>(p), b = *reinterpret_cast<const h4_t *>(p + 8);
        h8_t v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
        return v;
    };
    // k.k (waves 0, 1) and q.k of the three blocks of 32x32 on and below the diagonal: each wave has one of those with i in 32..63, and
    // half of the registers of the first on the diagonal, whose product both waves take.  They stay in registers, rows j for P
    // (lane = i, as its pages have it) and rows i for the others.
    const int which = wave >> 1, part = wave & 1;
    constexpr bool kByI = !BWD;                                           // of q.k
    const bool by_i = which && kByI;
    const auto product = [&](int ib, int jb) {
        acc_t x = zeros();
#pragma unroll
        for (int m = 0; m < 2 * DKB; ++m) {
            const h8_t a = row_page(which, 0, ib, m), b = row_page(0, 0, jb, m);
            x = by_i ? mfma(b, a, x) : mfma(a, b, x);
            if constexpr (PARTS == 2) {
                const h8_t al = row_page(which, 1, ib, m), bl = row_page(0, 1, jb, m);
                x = by_i ? mfma(bl, a, x) : mfma(a, bl, x);
                x = by_i ? mfma(b, al, x) : mfma(al, b, x);
            }
        }
        return x;
    };
    float prod[24];
    {
        const acc_t x = product(1, part);
#pragma unroll
        for (int r = 0; r < 16; ++r) prod[r] = x[r];
        const acc_t y = product(0, 0);
#pragma unroll
        for (int r = 0; r < 8; ++r) prod[16 + r] = part ? y[8 + r] : y[r];
    }
    {   // pages of keys and queries
        uint4 *out = ws.qk + (slot * d.H + hk) * ws.qk_pages * kPage + lane;
        constexpr int F = 4 * DKB;
        for (int i = wave; i < (BWD ? 4 : 2) * PARTS * F; i += 4) {
            const int kind = BWD ? i / (PARTS * F) : 2 * (i / (PARTS * F)), part = i / F % PARTS, f = i % F;      // K, KT, Q, QT
            h8_t v;
            if (!(kind & 1)) {
                v = row_page(kind >> 1, part, f / (2 * DKB), f % (2 * DKB));
            } else {                                                    // lane = dk; places 0..3 tokens 16 m + 4 half on, 4..7 those 8 on
                const _Float16 *p = &xs[kind >> 1][part][16 * (f % 4) + 4 * half][32 * (f / 4) + (lane & 16)];
                p += (lane & 15) / 4 * LD + 4 * (lane & 3);
                const h4_t a = read_columns(p), b = read_columns(p + 8 * LD);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
            }
            out[i * kPage] = __builtin_bit_cast(uint4, v);
        }
    }

    for (int hv = hk * d.group; hv < (hk + 1) * d.group; ++hv) {
        const int64_t rec = slot * d.Hv + hv;
        float *rows = ws.rows + rec * kRowsFloats;
        float *bt = betas[hv & 1];                                      // by turns: the last head's pages of T may still be on their way
        float ekb = 0.f;
        if (wave == 0) {
            double v = gv < -1e4f ? -1e4 : (double)gv;                  // a NaN stays
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const double t = __shfl_up(v, m);
                if (lane >= m) v += t;
            }
            v *= kLog2eD;
            const float E = decay_of(v, 0.0), F = decay_of(__shfl(v, 63), v);
            G[lane] = v;
            bt[lane] = b;
            const float ek = E * kap[0][lane];
            ekb = ek * b;
            rows[64 * (BWD ? kRowEKBack : kRowEK) + lane] = ek;
            rows[64 * kRowFK + lane] = F * kap[0][lane];
            rows[64 * kRowEQ + lane] = d.scale * E * kap[1][lane];
            if constexpr (BWD) {
                rows[64 * kRowBeta + lane] = b;
                rows[64 * kRowE + lane] = E;
                rows[64 * kRowF + lane] = F;
                rows[64 * kRowKK + lane] = kap[0][lane];
                rows[64 * kRowKQ + lane] = kap[1][lane];
                rows[64 * kRowSizeK + lane] = size[0][lane];
                rows[64 * kRowSizeQ + lane] = size[1][lane];
                reinterpret_cast<double *>(rows + 64 * kRowG)[lane] = v;
            }
            if (lane == 63) rows[kGamma] = E;
            if (hv + 1 < (hk + 1) * d.group) load_gates(hv + 1);
        }
        __syncthreads();                                                // also: keys and queries, or the last head's A and T, are free
        float val[24];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int ib = u ? 0 : 1, jb = u ? 0 : part;
            const int mine = 32 * (by_i ? ib : jb) + col;
            const double g_mine = G[mine];
            const float k_mine = kap[by_i ? 1 : 0][mine], k0 = fminf(k_mine, 1.f), k1 = fmaxf(k_mine, 1.f);
            float top = 0.f;
#pragma unroll
            for (int r = 0; r < (u ? 8 : 16); ++r) {
                const int other = 32 * (by_i ? jb : ib) + (u ? 16 * part : 0) + acc_row(r, half);
                const int i = by_i ? mine : other, j = by_i ? other : mine;
                const float D = by_i ? decay_of(g_mine, G[other]) : decay_of(G[other], g_mine);
                float x = prod[16 * u + r] * k0 * (kap[by_i ? 0 : which][other] * k1) * D * (which ? d.scale : bt[i]);
                asm("" : "+v"(x));                                      // all of it, then a selection: no branch for each
                x = j < i || (which && j == i) ? x : 0.f;
                val[16 * u + r] = x;
                top = fmaxf(top, fabsf(x));
                if (!which) A[i][j] = x;
            }
            top = max_halves(top);
            if (which && half == 0) top_p[part][u][col] = top;
        }
        __syncthreads();
        uint4 *out = ws.tri + rec * ws.tri_pages * kPage + lane;
        const auto put = [&](int kind, int page, const Pair &p) {
            out[((2 * kind) * kTriPages + page) * kPage] = __builtin_bit_cast(uint4, p.hi);
            out[((2 * kind + 1) * kTriPages + page) * kPage] = __builtin_bit_cast(uint4, p.lo);
        };
        if (which) {                                                    // P or P^T: registers 8 m .. 8 m + 7 are pages
            const auto page = [&](int ib, int jb, int m) { return BWD ? high_page(jb, 2 * ib + m) : low_page(ib, 2 * jb + m); };
            // the lane's row, which is in two tiles of P (rows 32.. and 0..31, the latter cut in two) or three or one of P^T
            const float first = fmaxf(top_p[0][1][col], top_p[1][1][col]);
            const float low = BWD ? fmaxf(first, top_p[0][0][col]) : first, high = BWD ? top_p[1][0][col] : fmaxf(top_p[0][0][col], top_p[1][0][col]);
            const float s_low = pow2_scale(low), s_high = pow2_scale(high), sp[2] = {BWD && !part ? s_low : s_high, s_low};
#pragma unroll
            for (int u = 0; u < 3; ++u)
                put(BWD ? 2 : 1, u < 2 ? page(1, part, u) : page(0, 0, part), split8(sp[u >> 1], [&](int e) { return val[8 * u + e]; }));
            if (part == 0) rows[64 * (BWD ? kRowInvPT : kRowInvP) + lane] = pow2_inv(half ? s_high : s_low);
        }

        // T: the blocks on the diagonal
        {
            const int o = 16 * wave, c = lane & 15;
            float t[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float v = i == c ? 1.f : 0.f;
#pragma unroll
                for (int j = 0; j < i; ++j) v = fmaf(-A[o + i][o + j], t[j], v);
                t[i] = v;
            }
            if (lane < 16) {
#pragma unroll
                for (int i = 0; i < 16; ++i) Ti[o + i][o + c] = t[i];
            }
        }
        __syncthreads();
        // and those below it: T_ij = -T_ii sum_k A_ik T_kj.  The contraction of step u takes elements 4 (lane/16) + u, the
        // rows in which a result lies in registers
#pragma unroll
        for (int lev = 1; lev < 4; ++lev) {
            if (wave < 4 - lev) {
                const int bi = wave + lev, bj = wave, c = lane & 15, o = 4 * (lane >> 4);
                f4_t sum = {0.f, 0.f, 0.f, 0.f}, res = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int kb = 0; kb < lev; ++kb)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        sum = __builtin_amdgcn_mfma_f32_16x16x4f32(A[16 * bi + c][16 * (bj + kb) + o + u],
                                                                   Ti[16 * (bj + kb) + o + u][16 * bj + c], sum, 0, 0, 0);
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    res = __builtin_amdgcn_mfma_f32_16x16x4f32(Ti[16 * bi + c][16 * bi + o + u], sum[u], res, 0, 0, 0);
#pragma unroll
                for (int u = 0; u < 4; ++u) Ti[16 * bi + o + u][16 * bj + c] = -res[u];
            }
            __syncthreads();
        }
        {
            float tm = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int i = tid >> 2, j = (tid & 3) * 16 + e;
                if (j <= i) tm = fmaxf(tm, fabsf(BWD ? Ti[i][j] : Ti[i][j] * bt[j]));
            }
            tm = fmaxf(tm, __shfl_xor(tm, 1));
            tm = fmaxf(tm, __shfl_xor(tm, 2));
            if ((tid & 3) == 0) top_t[tid >> 2] = tm;
            if constexpr (BWD) {
                tm = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int i = 16 * wave + e;
                    if (lane <= i) tm = fmaxf(tm, fabsf(Ti[i][lane]));
                }
                top_tt[wave][lane] = tm;
            }
        }
        __syncthreads();
        const auto scale_t = [&](int i) { return pow2_scale(top_t[i]); };
        const auto scale_tt = [&](int j) {
            constexpr int w = BWD ? 1 : 0;
            return pow2_scale(fmaxf(fmaxf(top_tt[0][j], top_tt[w][j]), fmaxf(top_tt[2 * w][j], top_tt[3 * w][j])));
        };
        if (wave == 0) {
            rows[64 * (BWD ? kRowInvTBack : kRowInvT) + lane] = pow2_inv(scale_t(lane));
            if constexpr (BWD) {
                const float inv = pow2_inv(scale_tt(lane));
                rows[64 * kRowInvTT + lane] = inv;
                rows[64 * kRowEZ + lane] = ekb * inv;
            }
        }
        for (int f = wave; f < kTriPages; f += 4) {
            const int ib = f < 2 ? 0 : 1, m = ib ? f - 2 : f, i = 32 * ib + col;
            const float st = scale_t(i);
            // forward: times beta of the column, so that the kernel behind it has R = V - E K S
            put(0, f, split8(st, [&](int e) {
                    const int j = page_at(m, half, e);
                    return j > i ? 0.f : BWD ? Ti[i][j] : Ti[i][j] * bt[j];
                }));
        }
        if constexpr (BWD) {
            for (int f = wave; f < kTriPages; f += 4) {
                const int jb = f < 4 ? 0 : 1, m = jb ? f - 2 : f, j = 32 * jb + col;
                const float st = scale_tt(j);
                put(1, f, split8(st, [&](int e) {
                        const int i = page_at(m, half, e);
                        return j <= i ? Ti[i][j] : 0.f;
                    }));
            }
        }
    }
}

__global__ __launch_bounds__(kThreads) void delta_fill_kernel(Seq s, Fill f) { fill_rows(s, f, blockIdx.x, gridDim.x); }

template <typename T, bool BWD>
void prep(const Seq &s, const Delta &d, const DeltaWs &ws, const DeltaIn &in, hipStream_t st) {
    const dim3 grid((unsigned)(ws.blocks * d.H));
#define CASE(n)                                                                                                               \
    case n:                                                                                                                   \
        delta_prep_kernel<T, n, BWD><<<grid, kThreads, 0, st>>>(s, d, ws, (const T *)in.q.p, in.q.ld, (const T *)in.k.p,       \
                                                                in.k.ld, (const float *)in.g.p, in.g.ld, (const float *)in.beta.p, \
                                                                in.beta.ld);                                                  \
        break
    switch ((d.Dk + 31) / 32) {
        CASE(1);
        CASE(2);
        CASE(3);
        CASE(4);
    }
#undef CASE
}

int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }

// Segments of a sequence: its chain of blocks is cut where there are too few chains to fill the chip's 1024 SIMDs with a wave
// each.  What a segment makes of any state is a matrix and an offset, found by running it from the identity and from zero
// (twice the columns); the segments are joined one after another, and run again from their states.  That is
// three times the work over n times the waves (one sequence of 32768 tokens in 8 heads of 128: 414 us; 2638 before there were segments).
// - Waves: packed sequences count as as many of the longest as hold their tokens (9 sequences of 5003 tokens, the longest of 2605,
//   fp32 in 6 heads of 72 and 99: 121 us, cut for nine of the longest 145).
// - A block takes 11 to 15 us in both passes and the joining of a segment 3: 2 sqrt(blocks) segments are the best number
//   (backward, 11981 tokens in 16 heads of 64 and 10: 478 us, with 47 segments instead of 27 505).
// - Fewer than three segments, or than eight blocks, do not pay (8 x 2048 tokens in 16 heads of 128 in two: forward 318 us
//   instead of 322, backward 950 instead of 914, at that step).
// - Every sequence's workgroups for every segment are launched, and end at once where it has none: at most 16384 waves.
void cut(const Seq &s, const Delta &d, DeltaWs &ws) {
    const int longest = (int)std::min<int64_t>(s.T, s.rows), blocks = (longest + kBlock - 1) / kBlock, slices = (d.Dv + 31) / 32;
    ws.segments = 1, ws.seg_blocks = std::max((s.T + kBlock - 1) / kBlock, 1);
    if (blocks < 8) return;
    const int64_t one = d.Hv * slices, waves = std::min<int64_t>(s.B, (s.rows + longest - 1) / longest) * one;
    const int n = (int)std::min({1024 / waves, (int64_t)blocks / 2, (int64_t)(2 * sqrt((double)blocks)), 16384 / (s.B * one)});
    if (n < 3) return;
    ws.seg_blocks = (blocks + n - 1) / n;
    ws.segments = (blocks + ws.seg_blocks - 1) / ws.seg_blocks;
}

// S' = M S + N from segment to segment: a workgroup to 32 columns, a wave to 32 rows of them.  M is loaded two
// segments ahead; S goes through LDS as pages, each wave's under its own powers of two, so that one barrier is all that a
// segment waits for.  N makes way for S'.
template <int DKB>
__global__ __launch_bounds__(64 * DKB) void delta_join_kernel(Seq s, Delta d, DeltaWs ws, int slices, bool back) {
    __shared__ __align__(16) h8_t pages[2][DKB][4][64];                 // by turns: of each wave, page 0 hi and lo, page 1 hi and lo
    __shared__ float inverse[2][DKB][32];
    const int lane = threadIdx.x & 63, half = lane >> 5, col = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int heads = s.B * d.Hv, bh = (int)(blockIdx.x % heads), slice = (int)(blockIdx.x / heads);
    int64_t first;
    int len;
    const int b = bh / d.Hv, hv = bh % d.Hv;
    seq_range(s, b, first, len);
    const int blocks = (len + kBlock - 1) / kBlock, n = (blocks + ws.seg_blocks - 1) / ws.seg_blocks;
    const int ld = 32 * slices, offset = 32 * DKB * ld, size = offset + 1024 * DKB * DKB;
    float *base = ws.sums + (first_segment(s, ws, b, first) * d.Hv + hv) * size;
    const uint32_t at = 4 * (32 * slice + col) + 32 * wave * 4 * ld;    // the wave's rows
    if (n < 3) return;
    const auto segment = [&](int i) { return base + (int64_t)(back ? n - 1 - i : i) * d.Hv * size; };
    // by turns, two segments ahead: the lane's row of M, in the order of a page's places, and N
    float row[2][16 * DKB];
    acc_t S[1], N[1], next[2][1];
    const auto fetch = [&](int i, float(&r)[16 * DKB], acc_t(&to)[1]) {
        const float *p = segment(i) + offset + 32 * wave + col + 4 * half * 32 * DKB;
#pragma unroll
        for (int u = 0; u < 16 * DKB; ++u) r[u] = p[page_at(u >> 3, 0, u & 7) * 32 * DKB];
        load_state<1>(make_rsrc(segment(i), 4 * offset), at, 4 * ld, half, to);
    };
    load_state<1>(make_rsrc(segment(0), 4 * offset), at, 4 * ld, half, S);
    fetch(1, row[1], next[1]);
    if (n > 3) fetch(2, row[0], next[0]);
    const auto step = [&](int i, auto turn) {
        constexpr int x = decltype(turn)::value;
        float m = 0.f;
#pragma unroll
        for (int u = 0; u < 16 * DKB; ++u) m = fmaxf(m, fabsf(row[x][u]));
#pragma unroll
        for (int u = 1; u < 64; u <<= 1) m = fmaxf(m, __shfl_xor(m, u));
        const float sm = pow2_scale(m), im = pow2_inv(sm);
        Pair w[2 * DKB];
#pragma unroll
        for (int u = 0; u < 2 * DKB; ++u) w[u] = split8(sm, [&](int j) { return row[x][8 * u + j]; });
        N[0] = next[x][0];
        if (i + 2 < n - 1) fetch(i + 2, row[x], next[x]);
        const float sc = pow2_scale(max_halves(max_abs(S[0])));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const Pair f = split8(sc, [&](int j) { return S[0][8 * u + j]; });
            pages[x][wave][2 * u][lane] = f.hi;
            pages[x][wave][2 * u + 1][lane] = f.lo;
        }
        if (half == 0) inverse[x][wave][col] = pow2_inv(sc);
        __syncthreads();
#pragma unroll
        for (int q = 0; q < DKB; ++q) {
            acc_t a = zeros();
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const h8_t hi = pages[x][q][2 * u][lane], lo = pages[x][q][2 * u + 1][lane];
                a = mfma(w[2 * q + u].hi, hi, a);
                a = mfma(w[2 * q + u].hi, lo, a);
                a = mfma(w[2 * q + u].lo, hi, a);
            }
            const float f = inverse[x][q][col];
#pragma unroll
            for (int j = 0; j < 16; ++j) N[0][j] = fmaf(a[j] * im, f, N[0][j]);
        }
        S[0] = N[0];
        store_state<1>(make_rsrc(segment(i), 4 * offset), at, 4 * ld, half, S);
    };
    for (int i = 1; i < n - 1; i += 2) {
        step(i, std::integral_constant<int, 1>());
        if (i + 1 < n - 1) step(i + 1, std::integral_constant<int, 0>());
    }
}

}  // namespace

hipError_t launch_delta_join(const Seq &s, const Delta &d, const DeltaWs &ws, bool back, hipStream_t st) {
    const int slices = (d.Dv + 31) / 32;
    const unsigned grid = (unsigned)(s.B * d.Hv * slices);
    switch ((d.Dk + 31) / 32) {
    case 1: delta_join_kernel<1><<<grid, 64, 0, st>>>(s, d, ws, slices, back); break;
    case 2: delta_join_kernel<2><<<grid, 128, 0, st>>>(s, d, ws, slices, back); break;
    case 3: delta_join_kernel<3><<<grid, 192, 0, st>>>(s, d, ws, slices, back); break;
    default: delta_join_kernel<4><<<grid, 256, 0, st>>>(s, d, ws, slices, back);
    }
    return hipGetLastError();
}

int64_t delta_layout(const Seq &s, const Delta &d, bool bf16, bool bwd, void *base, DeltaWs &ws) {
    const int dkb = (d.Dk + 31) / 32, dvb = (d.Dv + 31) / 32;
    ws.per = (s.T + kBlock - 1) / kBlock;
    ws.blocks = s.off ? s.rows / kBlock + s.B : (int64_t)s.B * ws.per;
    ws.qk_pages = (bwd ? 4 : 2) * (bf16 ? 1 : 2) * 4 * dkb;
    ws.tri_pages = (bwd ? 6 : 4) * kTriPages;
    char *p = (char *)base;
    int64_t at = 0;
    const auto take = [&](int64_t bytes) {
        char *r = p + at;
        at += round16(bytes);
        return r;
    };
    ws.qk = (uint4 *)take(ws.blocks * d.H * ws.qk_pages * 1024);
    ws.tri = (uint4 *)take(ws.blocks * d.Hv * ws.tri_pages * 1024);
    ws.rows = (float *)take(ws.blocks * d.Hv * kRowsFloats * 4);
    ws.ends = bwd ? (float *)take(ws.blocks * d.Hv * dkb * dvb * 4096) : nullptr;
    cut(s, d, ws);
    const int64_t segments = s.off ? s.rows / ((int64_t)kBlock * ws.seg_blocks) + s.B : (int64_t)s.B * ws.segments;
    ws.sums = ws.segments > 1 ? (float *)take(segments * d.Hv * dkb * (dkb + dvb) * 4096) : nullptr;
    return at;
}

void launch_delta_prep(const Seq &s, const Delta &d, bool bf16, bool bwd, const DeltaWs &ws, const DeltaIn &in, const Fill &fill, hipStream_t st) {
    // a launch of its own (4.5 us): workgroups of the kernel below in its place made that one slower for everybody (122 to 154 us)
    if (fill.blocks) delta_fill_kernel<<<fill.blocks, kThreads, 0, st>>>(s, fill);
    if (bf16) bwd ? prep<uint16_t, true>(s, d, ws, in, st) : prep<uint16_t, false>(s, d, ws, in, st);
    else bwd ? prep<float, true>(s, d, ws, in, st) : prep<float, false>(s, d, ws, in, st);
}

}  // namespace convfwd
