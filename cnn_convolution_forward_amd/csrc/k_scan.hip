// k_scan.hip -- the gated linear recurrence over tokens: forward, backward and
// the single-token step (conv_scan_*).
#include "conv_fwd.h"
#include "scan_math.h"

namespace convfwd {
namespace {

constexpr int kBlock = CONV_SCAN_BLOCK;
constexpr int kWaves = 8, kThreads = 64 * kWaves;

// ---- chunks and the carries between them -----------------------------------------
//
// The recurrence is a chain of affine maps h -> A h + H, so a chunk of tokens
// composes into one map before the state in front of it is known.  A workgroup
// takes one chunk of 64 * VEC channels; its waves take consecutive tokens, kept
// in registers from the only read of the inputs.  It publishes its map, obtains
// the state in front of it, publishes the state behind it, and then runs its
// tokens.
//
// The state in front of chunk k: the nearest predecessor that has published its
// outgoing state, carried through the maps of those between.  Each step of that
// fold is c = fma(A, c, H), the operation by which the predecessor itself makes
// its outgoing state, so the result does not depend on where the fold starts:
// bits do not depend on timing.
//
// Waits end: workgroups take their chunk from a counter, chunks of a sequence
// in order, so every predecessor is held by a workgroup that is running or
// done, and the lowest unfinished one waits for nobody.  A published word is its
// own flag: the workspace is filled with ones (a NaN that is never stored)
// first, and words are written and read whole by relaxed atomics of device
// scope, so nothing else has to be ordered.  The poll count is bounded all the
// same; running out gives NaN.

constexpr uint32_t kEmpty = 0xffffffffu;
constexpr int kMaxPolls = 1 << 22;

__device__ __forceinline__ uint32_t word(float v) {
    const uint32_t u = __float_as_uint(v);
    return u == kEmpty ? 0x7fc00000u : u;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) { return (uint64_t)word(lo) | (uint64_t)word(hi) << 32; }
__device__ __forceinline__ float low(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float high(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
template <typename W> __device__ __forceinline__ void put(W *p, W v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename W> __device__ __forceinline__ W get(const W *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Chunks are blocks of `tokens` tokens (packed_block numbers them).
struct Chunks {
    int tokens, per;
    int64_t total;
    uint32_t *counter;
    int32_t *off;           // offsets clamped to [0, rows] and made to ascend
    uint64_t *map;          // (total, C): A, H
    uint32_t *state;        // (total, C): state behind the chunk
};

struct Tile {
    int b, k, ct;           // sequence, chunk in it (negative: an unused number), block of channels
    int64_t slot;           // number of the chunk
};

// REV: later chunks of a sequence first.
template <bool REV> __device__ __forceinline__ Tile get_tile(const Seq &s, const Chunks &ch, int nct, uint32_t ticket) {
    Tile t;
    t.ct = ticket % nct;
    const int64_t rest = ticket / nct;
    if (!s.off || ch.per == 1) {
        t.b = (int)(rest % s.B);
        const int k = (int)(rest / s.B);
        t.k = REV ? ch.per - 1 - k : k;
        t.slot = (int64_t)t.b * ch.per + t.k;
    } else {
        t.slot = REV ? ch.total - 1 - rest : rest;
        const Block k = packed_block(s, ch.tokens, t.slot);
        t.b = k.b;
        t.k = k.k;
    }
    return t;
}

__device__ __forceinline__ uint32_t take_ticket(uint32_t *counter, uint32_t *shared) {
    if (threadIdx.x == 0) *shared = atomicAdd(counter, 1u);
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(*shared);
}

// The state that reaches chunk `slot` from the chunks at slot + dir, slot + 2 dir, ... (nearest first;
// `n` of them, the last of which publishes its state without waiting).  One wave; lanes beyond the
// channels hold a valid column.
template <int VEC>
__device__ __forceinline__ void carry_in(const Chunks &ch, int C, int c, int64_t slot, int dir, int n, float (&h)[VEC]) {
    constexpr int kAhead = 4;
    const uint64_t *maps = ch.map + slot * C + c;
    const uint32_t *states = ch.state + slot * C + c;
    const int64_t step = (int64_t)dir * C;
    int at = 1, polls = 0, found = 0;
    uint32_t st[kAhead][VEC];
    while (!found) {
        uint64_t mp[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t o = (int64_t)min(at + i, n) * step;
#pragma unroll
            for (int v = 0; v < VEC; ++v) st[i][v] = get(states + o + v);
            mp[i] = get(maps + o + VEC - 1);
            if (VEC > 1 && (uint32_t)get(maps + o) == kEmpty) mp[i] = kEmpty;
        }
        int moved = 0;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            bool ready = true;
#pragma unroll
            for (int v = 0; v < VEC; ++v) ready = ready && st[i][v] != kEmpty;
            if (!found && moved == i && at + i <= n) {
                if (__all(ready)) {
                    found = at + i;
#pragma unroll
                    for (int v = 0; v < VEC; ++v) h[v] = __uint_as_float(st[i][v]);
                } else if (at + i < n && __all((uint32_t)mp[i] != kEmpty)) {
                    ++moved;
                }
            }
        }
        at += moved;
        if (!found && !moved) {
            if (++polls > kMaxPolls) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) h[v] = __uint_as_float(0x7fc00000u);
                return;
            }
            __builtin_amdgcn_s_sleep(1);
        }
    }
    for (int i = found - 1; i >= 1; i -= kAhead) {
        uint64_t mp[kAhead][VEC];
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
#pragma unroll
            for (int v = 0; v < VEC; ++v) mp[q][v] = get(maps + (int64_t)max(i - q, 1) * step + v);
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
            if (i - q >= 1) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) h[v] = fmaf(low(mp[q][v]), h[v], high(mp[q][v]));
            }
    }
}

// Empties the links, and (block 0, packed sequences) makes the offsets ascend.
__global__ __launch_bounds__(256) void scan_fill_kernel(Seq s, Chunks ch, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) reinterpret_cast<uint4 *>(ch.map)[i] = make_uint4(kEmpty, kEmpty, kEmpty, kEmpty);
    if (i == 0) *ch.counter = 0;
    if (s.off && blockIdx.x == 0 && threadIdx.x < 64) {
        int most = 0;
        for (int base = 0; base <= s.B; base += 64) {
            const int j = base + (int)threadIdx.x;
            int v = j <= s.B ? (int)min((int64_t)max(s.off[j], 0), s.rows) : 0;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int u = __shfl_up(v, o);
                if ((int)threadIdx.x >= o) v = max(v, u);
            }
            v = max(v, most);
            if (j <= s.B) ch.off[j] = v;
            most = __shfl(v, 63);
        }
    }
}

// ---- forward -----------------------------------------------------------------------

constexpr int kFwdRun = 16, kFwdChunk = kWaves * kFwdRun;      // tokens of a wave and of a workgroup

template <typename T, int VEC, bool CHAIN>
__global__ __launch_bounds__(kThreads, 4) void scan_fwd_kernel(
    Seq s, float scale, const T *__restrict__ x, int64_t ldx, const T *__restrict__ gate, int64_t ldg,
    const T *__restrict__ inp, int64_t ldi, const float *__restrict__ decay, const float *__restrict__ h0,
    T *__restrict__ y, int64_t ldy, float *__restrict__ hT, float *__restrict__ states, Chunks ch, int nct) {
    constexpr int L = kFwdRun, CW = 64 * VEC;
    __shared__ float sA[kWaves][CW], sH[kWaves][CW], sC[CW];
    __shared__ uint32_t sTicket;
    const Tile tile = get_tile<false>(s, ch, nct, CHAIN ? take_ticket(ch.counter, &sTicket) : blockIdx.x);
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int b = tile.b, C = s.C;
    int64_t first;
    int len;
    seq_range(s, b, first, len);
    const int t0 = tile.k * kFwdChunk;
    if (tile.k < 0 || (t0 >= len && tile.k > 0)) return;
    const int cw = tile.ct * CW + lane * VEC;
    const bool on = cw < C;
    const int c = min(cw, C - VEC);                // odd C: the last lane shares a channel, with the same results
    const int tw = t0 + w * L;                     // this wave's tokens: tw .. min(tw + L, len)
    float k[VEC], a[L][VEC], bb[L][VEC], A[VEC], H[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) A[v] = 1.f, H[v] = 0.f;
    if (tw < len) {
        typename Pack<T, VEC>::type xr[L], gr[L], ir[L];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int64_t row = first + min(tw + i, len - 1);
            gr[i] = load_pack<T, VEC>(gate + row * ldg + c);
            ir[i] = load_pack<T, VEC>(inp + row * ldi + c);
            xr[i] = load_pack<T, VEC>(x + row * ldx + c);
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) k[v] = scan_rate(scale, decay[c + v]);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            float xv[VEC], gv[VEC], iv[VEC];
            to_f32(xr[i], xv);
            to_f32(gr[i], gv);
            to_f32(ir[i], iv);
            const bool in = tw + i < len;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const ScanGates g(k[v], gv[v], iv[v]);
                a[i][v] = in ? g.a : 1.f;
                bb[i][v] = in ? g.m * g.s * xv[v] : 0.f;
                A[v] *= a[i][v];
                H[v] = fmaf(a[i][v], H[v], bb[i][v]);
            }
        }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) sA[w][lane * VEC + v] = A[v], sH[w][lane * VEC + v] = H[v];
    __syncthreads();
    float PA[VEC], PH[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) PA[v] = 1.f, PH[v] = 0.f;
    for (int q = 0; q < w; ++q)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float Aq = sA[q][lane * VEC + v], Hq = sH[q][lane * VEC + v];
            PH[v] = fmaf(Aq, PH[v], Hq);
            PA[v] *= Aq;
        }
    if (w == kWaves - 1) {                       // this wave has the whole chunk's map
        float c0[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            H[v] = fmaf(A[v], PH[v], H[v]);
            A[v] *= PA[v];
        }
        const bool last = !CHAIN || t0 + kFwdChunk >= len;
        const int64_t at = tile.slot * C + c;
        if (tile.k == 0) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) c0[v] = h0 ? h0[(int64_t)b * C + c + v] : 0.f;
        } else if (CHAIN) {
            if (!last && on)
#pragma unroll
                for (int v = 0; v < VEC; ++v) put(ch.map + at + v, pair(A[v], H[v]));
            carry_in<VEC>(ch, C, c, tile.slot, -1, tile.k, c0);
        }
        if (!last && on)
#pragma unroll
            for (int v = 0; v < VEC; ++v) put(ch.state + at + v, word(fmaf(A[v], c0[v], H[v])));
#pragma unroll
        for (int v = 0; v < VEC; ++v) sC[lane * VEC + v] = c0[v];
    }
    __syncthreads();
    float h[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = fmaf(PA[v], sC[lane * VEC + v], PH[v]);
    if (!on) return;
    if (tw < len) {
        if (states && tw % kBlock == 0) {
            const int64_t nb = (s.T + kBlock - 1) / kBlock;
#pragma unroll
            for (int v = 0; v < VEC; ++v) states[(b * nb + tw / kBlock) * C + c + v] = h[v];
        }
#pragma unroll
        for (int i = 0; i < L; ++i) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) h[v] = fmaf(a[i][v], h[v], bb[i][v]);
            if (tw + i < len) store_f32(y + (first + tw + i) * ldy + c, h);
        }
        if (hT && tw + L >= len)
#pragma unroll
            for (int v = 0; v < VEC; ++v) hT[(int64_t)b * C + c + v] = h[v];
    } else if (hT && len == 0 && w == 0) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) hT[(int64_t)b * C + c + v] = h[v];
    }
}

// ---- backward ----------------------------------------------------------------------
//
// e[t] = a[t] dh[t] is what the gradient of h[t-1] receives: e_in -> a (dy + e_in)
// is affine with the same factor, so the chunks chain as in the forward pass, the
// other way round.  h[t-1] is run forward again from the saved state at the
// chunk's start, in the same pass over the registers.

constexpr int kBwdRun = 8, kBwdChunk = kWaves * kBwdRun;
static_assert(kBwdChunk == kBlock, "a saved state for every chunk");

template <typename T, int VEC, bool CHAIN>
__global__ __launch_bounds__(kThreads, 4) void scan_bwd_kernel(
    Seq s, float scale, const T *__restrict__ x, int64_t ldx, const T *__restrict__ gate, int64_t ldg,
    const T *__restrict__ inp, int64_t ldi, const float *__restrict__ decay, const float *__restrict__ states,
    const T *__restrict__ dy, int64_t lddy, const float *__restrict__ dhT, T *__restrict__ dx, int64_t lddx,
    T *__restrict__ dgate, int64_t lddg, T *__restrict__ dinp, int64_t lddi, float *__restrict__ part,
    float *__restrict__ dh0, Chunks ch, int nct) {
    constexpr int L = kBwdRun, CW = 64 * VEC;
    __shared__ float sA[kWaves][CW], sH[kWaves][CW], sE[kWaves][CW], sC[CW];
    __shared__ uint32_t sTicket;
    const Tile tile = get_tile<true>(s, ch, nct, CHAIN ? take_ticket(ch.counter, &sTicket) : blockIdx.x);
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int b = tile.b, C = s.C;
    int64_t first;
    int len;
    seq_range(s, b, first, len);
    const int t0 = tile.k * kBwdChunk;
    const int cw = tile.ct * CW + lane * VEC;
    const bool on = cw < C;
    const int c = min(cw, C - VEC);                // odd C: the last lane shares a channel, with the same results
    if (tile.k < 0 || t0 >= len) {                // an unused number, or an empty sequence
        if (on && w == 0)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                part[tile.slot * C + c + v] = 0.f;
                if (len == 0 && tile.k == 0 && dh0)
                    dh0[(int64_t)b * C + c + v] = dhT ? dhT[(int64_t)b * C + c + v] : 0.f;
            }
        return;
    }
    const int tw = t0 + w * L;
    float k[VEC], A[VEC], H[VEC], E[VEC];
    float a[L][VEC], r[L][VEC], sg[L][VEC], im[L][VEC], m[L][VEC];
    typename Pack<T, VEC>::type xr[L], gr[L], ir[L], dr[L];
#pragma unroll
    for (int v = 0; v < VEC; ++v) A[v] = 1.f, H[v] = 0.f, E[v] = 0.f;
    if (tw < len) {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int64_t row = first + min(tw + i, len - 1);
            gr[i] = load_pack<T, VEC>(gate + row * ldg + c);
            ir[i] = load_pack<T, VEC>(inp + row * ldi + c);
            xr[i] = load_pack<T, VEC>(x + row * ldx + c);
            dr[i] = load_pack<T, VEC>(dy + row * lddy + c);
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) k[v] = scan_rate(scale, decay[c + v]);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            float xv[VEC], gv[VEC], iv[VEC];
            to_f32(xr[i], xv);
            to_f32(gr[i], gv);
            to_f32(ir[i], iv);
            const bool in = tw + i < len;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const ScanGates g(k[v], gv[v], iv[v]);
                a[i][v] = in ? g.a : 1.f;
                r[i][v] = g.r, sg[i][v] = g.s, im[i][v] = g.im, m[i][v] = in ? g.m : 0.f;
                A[v] *= a[i][v];
                H[v] = fmaf(a[i][v], H[v], in ? g.m * g.s * xv[v] : 0.f);
            }
        }
#pragma unroll
        for (int i = L - 1; i >= 0; --i) {
            float dv[VEC];
            to_f32(dr[i], dv);
#pragma unroll
            for (int v = 0; v < VEC; ++v) E[v] = a[i][v] * (tw + i < len ? dv[v] + E[v] : E[v]);
        }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v)
        sA[w][lane * VEC + v] = A[v], sH[w][lane * VEC + v] = H[v], sE[w][lane * VEC + v] = E[v];
    __syncthreads();
    // h in front of this wave's tokens; the map from the chunk's e_in to this wave's
    float h[VEC], PA[VEC], PE[VEC];
    const int64_t nb = (s.T + kBlock - 1) / kBlock;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        h[v] = states[(b * nb + tile.k) * C + c + v];
        PA[v] = 1.f, PE[v] = 0.f;
    }
    for (int q = 0; q < w; ++q)
#pragma unroll
        for (int v = 0; v < VEC; ++v) h[v] = fmaf(sA[q][lane * VEC + v], h[v], sH[q][lane * VEC + v]);
    for (int q = kWaves - 1; q > w; --q)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float Aq = sA[q][lane * VEC + v];
            PE[v] = fmaf(Aq, PE[v], sE[q][lane * VEC + v]);
            PA[v] *= Aq;
        }
    if (w == 0) {
        float c0[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            E[v] = fmaf(A[v], PE[v], E[v]);
            A[v] *= PA[v];
        }
        const int behind = (len + kBwdChunk - 1) / kBwdChunk - 1 - tile.k;       // chunks after this one
        const int64_t at = tile.slot * C + c;
        if (!CHAIN || behind == 0) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) c0[v] = dhT ? dhT[(int64_t)b * C + c + v] : 0.f;
        } else {
            if (tile.k > 0 && on)
#pragma unroll
                for (int v = 0; v < VEC; ++v) put(ch.map + at + v, pair(A[v], E[v]));
            carry_in<VEC>(ch, C, c, tile.slot, 1, behind, c0);
        }
        if (on)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float out = fmaf(A[v], c0[v], E[v]);
                if (CHAIN && tile.k > 0) put(ch.state + at + v, word(out));
                if (dh0 && tile.k == 0) dh0[(int64_t)b * C + c + v] = out;
            }
#pragma unroll
        for (int v = 0; v < VEC; ++v) sC[lane * VEC + v] = c0[v];
    }
    __syncthreads();
    float dk[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) dk[v] = 0.f;
    if (tw < len) {
        float e[VEC], before[L][VEC];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            float xv[VEC];
            to_f32(xr[i], xv);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                before[i][v] = h[v];
                h[v] = fmaf(a[i][v], h[v], m[i][v] * sg[i][v] * xv[v]);
            }
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) e[v] = fmaf(PA[v], sC[lane * VEC + v], PE[v]);
#pragma unroll
        for (int i = L - 1; i >= 0; --i) {
            if (tw + i >= len) continue;
            float xv[VEC], dv[VEC], o0[VEC], o1[VEC], o2[VEC];
            to_f32(xr[i], xv);
            to_f32(dr[i], dv);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float dh = dv[v] + e[v], dms = dh * m[i][v] * sg[i][v];
                const float dla = dh * a[i][v] * (before[i][v] - sg[i][v] * xv[v] * a[i][v] * im[i][v]);
                const float rdla = r[i][v] * dla;
                o0[v] = dms;
                o1[v] = -k[v] * rdla * (1.f - r[i][v]);
                o2[v] = dms * xv[v] * (1.f - sg[i][v]);
                dk[v] += rdla;
                e[v] = a[i][v] * dh;
            }
            if (on) {
                const int64_t row = first + tw + i;
                store_f32(dx + row * lddx + c, o0);
                store_f32(dgate + row * lddg + c, o1);
                store_f32(dinp + row * lddi + c, o2);
            }
        }
    }
    // sA is free: every wave read it before the barrier above
#pragma unroll
    for (int v = 0; v < VEC; ++v) sA[w][lane * VEC + v] = dk[v];
    __syncthreads();
    if (w == 0 && on)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float d = 0.f;
            for (int q = 0; q < kWaves; ++q) d += sA[q][lane * VEC + v];
            part[tile.slot * C + c + v] = d;
        }
}

// ddecay[c] = -scale sigmoid(decay) * the sum of the chunks' partial sums: 16
// channels per workgroup, 64 strands of rows, each added in order.
__global__ __launch_bounds__(1024) void scan_reduce_kernel(const float *__restrict__ part, int64_t n, int C, float scale,
                                                           const float *__restrict__ decay, float *__restrict__ ddecay) {
    __shared__ float red[64][17];
    const int cl = threadIdx.x & 15, q = threadIdx.x >> 4, c = blockIdx.x * 16 + cl;
    float v = 0.f;
    if (c < C)
        for (int64_t i = q; i < n; i += 64) v += part[i * C + c];
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
        ddecay[c] = -scale * sigmoid(decay[c]) * v;
    }
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

Chunks chunks(const Seq &s, int tokens) {
    Chunks ch = {};
    ch.tokens = tokens;
    ch.per = s.T > 0 ? (s.T + tokens - 1) / tokens : 1;
    ch.total = block_count(s, tokens, ch.per);
    return ch;
}

// Workspace of the links: the counter (16 bytes), the offsets, then per chunk and channel 8 bytes of
// map and 4 of state, each part to a multiple of 16; none if no sequence has a second chunk.
int64_t off_bytes(const Seq &s) { return s.off ? ((int64_t)s.B + 4) / 4 * 16 : 0; }
int64_t link_units(const Seq &s, const Chunks &ch) { return (ch.total * s.C * 12 + 15) / 16; }
size_t link_bytes(const Seq &s, const Chunks &ch) {
    return ch.per > 1 ? (size_t)(16 + off_bytes(s) + 16 * link_units(s, ch)) : 0;
}

// Lays the links out in ws and empties them; s then has the ascending offsets.
void set_links(Seq &s, Chunks &ch, void *ws, hipStream_t st) {
    if (ch.per <= 1) return;
    ch.counter = (uint32_t *)ws;
    ch.off = (int32_t *)((char *)ws + 16);
    ch.map = (uint64_t *)((char *)ws + 16 + off_bytes(s));
    ch.state = (uint32_t *)(ch.map + ch.total * s.C);
    const int64_t n = link_units(s, ch);
    scan_fill_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(s, ch, n);
    if (s.off) s.off = ch.off;
}

}  // namespace

size_t scan_fwd_workspace(const Seq &s) { return link_bytes(s, chunks(s, kFwdChunk)); }
size_t scan_bwd_workspace(const Seq &s) {
    const Chunks ch = chunks(s, kBwdChunk);
    return link_bytes(s, ch) + (size_t)ch.total * s.C * sizeof(float);
}

template <typename T, int VEC>
static void scan_fwd(const Seq &s, float scale, const void *x, int64_t ldx, const void *gate, int64_t ldg, const void *inp,
                     int64_t ldi, const float *decay, const float *h0, void *y, int64_t ldy, float *hT, float *states,
                     Chunks ch, hipStream_t st) {
    const int nct = (s.C + 64 * VEC - 1) / (64 * VEC);
    const unsigned grid = (unsigned)(ch.total * nct);
    if (ch.per > 1)
        scan_fwd_kernel<T, VEC, true><<<grid, kThreads, 0, st>>>(s, scale, (const T *)x, ldx, (const T *)gate, ldg,
                                                                 (const T *)inp, ldi, decay, h0, (T *)y, ldy, hT, states, ch, nct);
    else
        scan_fwd_kernel<T, VEC, false><<<grid, kThreads, 0, st>>>(s, scale, (const T *)x, ldx, (const T *)gate, ldg,
                                                                  (const T *)inp, ldi, decay, h0, (T *)y, ldy, hT, states, ch, nct);
}

hipError_t launch_scan_fwd(const Seq &s, bool bf16, float scale, const void *x, int64_t ldx, const void *gate,
                           int64_t ldg, const void *inp, int64_t ldi, const float *decay, const float *h0, void *y,
                           int64_t ldy, float *hT, float *states, void *ws, hipStream_t st) {
    Chunks ch = chunks(s, kFwdChunk);
    Seq q = s;
    set_links(q, ch, ws, st);
    const auto run = !bf16 ? scan_fwd<float, 1> : s.C > 1 ? scan_fwd<uint16_t, 2> : scan_fwd<uint16_t, 1>;
    run(q, scale, x, ldx, gate, ldg, inp, ldi, decay, h0, y, ldy, hT, states, ch, st);
    return hipGetLastError();
}

template <typename T, int VEC>
static void scan_bwd(const Seq &s, float scale, const void *x, int64_t ldx, const void *gate, int64_t ldg, const void *inp,
                     int64_t ldi, const float *decay, const float *states, const void *dy, int64_t lddy, const float *dhT,
                     void *dx, int64_t lddx, void *dgate, int64_t lddg, void *dinp, int64_t lddi, float *part, float *dh0,
                     Chunks ch, hipStream_t st) {
    const int nct = (s.C + 64 * VEC - 1) / (64 * VEC);
    const unsigned grid = (unsigned)(ch.total * nct);
    if (ch.per > 1)
        scan_bwd_kernel<T, VEC, true><<<grid, kThreads, 0, st>>>(
            s, scale, (const T *)x, ldx, (const T *)gate, ldg, (const T *)inp, ldi, decay, states, (const T *)dy, lddy, dhT,
            (T *)dx, lddx, (T *)dgate, lddg, (T *)dinp, lddi, part, dh0, ch, nct);
    else
        scan_bwd_kernel<T, VEC, false><<<grid, kThreads, 0, st>>>(
            s, scale, (const T *)x, ldx, (const T *)gate, ldg, (const T *)inp, ldi, decay, states, (const T *)dy, lddy, dhT,
            (T *)dx, lddx, (T *)dgate, lddg, (T *)dinp, lddi, part, dh0, ch, nct);
}

hipError_t launch_scan_bwd(const Seq &s, bool bf16, float scale, const void *x, int64_t ldx, const void *gate, int64_t ldg,
                           const void *inp, int64_t ldi, const float *decay, const float *states, const void *dy, int64_t lddy,
                           const float *dhT, void *dx, int64_t lddx, void *dgate, int64_t lddg, void *dinp, int64_t lddi,
                           float *ddecay, float *dh0, void *ws, hipStream_t st) {
    Chunks ch = chunks(s, kBwdChunk);
    Seq q = s;
    set_links(q, ch, ws, st);
    float *part = (float *)((char *)ws + link_bytes(s, ch));
    const auto run = !bf16 ? scan_bwd<float, 1> : s.C > 1 ? scan_bwd<uint16_t, 2> : scan_bwd<uint16_t, 1>;
    run(q, scale, x, ldx, gate, ldg, inp, ldi, decay, states, dy, lddy, dhT, dx, lddx, dgate, lddg, dinp, lddi, part, dh0, ch,
        st);
    scan_reduce_kernel<<<(s.C + 15) / 16, 1024, 0, st>>>(part, ch.total, s.C, scale, decay, ddecay);
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
