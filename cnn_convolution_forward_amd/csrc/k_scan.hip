// k_scan.hip -- the gated linear recurrence over tokens: forward, backward and
// the single-token step (conv_scan_*).
//
// HBM is the bound: forward reads x and two gates and writes y, backward reads
// those and dy and writes three gradients, each once; the arithmetic of the gates
// (six transcendental and about 28 other instructions an element forward) takes
// half of that time, counted by SQ_ACTIVE_INST_VALU.  Measured at 8 x 2048 x 2048
// bf16: forward 62.7 us, 4.3 TB/s (52 us at the rate of a large copy, 5.2 TB/s);
// backward 108.3 us, 4.4 TB/s, with 4 to 5 us each in the kernel before it and the
// one behind; one sequence of 32768 x 1024 forward 78 us, 3.4 TB/s.  A thread per
// sequence and channel, walking its tokens, took 1064, 2044 and 16454 us.
#include <algorithm>
#include <type_traits>

#include "conv_fwd.h"
#include "scan_grid.h"
#include "scan_math.h"

namespace convfwd {
namespace {

constexpr int kBlock = CONV_SCAN_BLOCK;
constexpr int kWaves = 8, kThreads = 64 * kWaves;
static_assert(kThreads == kScanThreads, "the grid is limited by its threads");

// ---- chunks and the carries between them -----------------------------------------
//
// The recurrence is a chain of affine maps h -> A h + H, so a chunk of tokens
// composes into one map before the state in front of it is known.  A workgroup
// takes one chunk of 64 * VEC channels; its waves take consecutive tokens, kept
// in registers from the only read of the inputs.  It publishes its map, obtains
// the state in front of it, publishes the state behind it, and then runs its
// tokens.  (Published as the single-pass scan with look-back: D. Merrill, M. Garland, 2016;
// here the elements are affine maps, and what is folded is the state itself.)
//
// The state in front of chunk k: the nearest predecessor that has published its
// outgoing state, carried through the maps of those between.  Each step of that
// fold is c = fma(A, c, H), the operation by which the predecessor itself makes
// its outgoing state, so the result does not depend on where the fold starts:
// bits do not depend on timing.
//
// Waits end: workgroups take their chunk from a counter, chunks of a sequence
// in order, so every predecessor is held by a workgroup that is running or
// done, and the lowest unfinished one waits for nobody.  One counter for all
// would be the bound: adds to one address follow each other at about 18 ns, 2048
// chunks of the training batch 37 us; so there are some 64, each with blocks of
// channels and sequences of its own, and a workgroup's index says which it uses.
// The poll count is bounded all the same; running out gives NaN.
//
// A published word is its own flag: the workspace is filled with ones (a NaN that
// is never stored) first, and words are written and read whole by relaxed atomics
// of device scope, so nothing else has to be ordered.  One more word per chunk and
// block of channels says how far it is; it only tells 64 lanes where to look, at
// 64 chunks in one load.
//
// Workgroups that keep taking chunks, with the next chunk's rows or only its
// ticket ahead, were slower (105 and 76 us against 65 at 8 x 2048 x 2048): loads
// return in order, so polls wait for rows under way, and a workgroup that ends
// makes room for one that starts while its stores drain.

constexpr uint32_t kEmpty = 0xffffffffu;
constexpr int kMaxPolls = 1 << 22;
enum : uint32_t { kNothing = 0, kMap = 1, kState = 2 };

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
    int tokens, per, nct;   // nct: blocks of channels
    int groups, nb;         // counters (a multiple of nct), sequences of each
    int64_t total;
    uint32_t *counter;      // kCounter apart
    int32_t *off;           // offsets clamped to [0, rows] and made to ascend
    float *rate;            // (C): k
    uint32_t *stage;        // (total, nct): kNothing, kMap, kState
    uint64_t *map;          // (total, C): A, H
    uint32_t *state;        // (total, C): state behind the chunk
};

constexpr int kCounter = 16;        // words: a counter has 64 bytes to itself

struct Tile {
    int b, k, ct;           // sequence, chunk in it (negative: an unused number), block of channels
    int64_t slot;           // number of the chunk; negative: there is none
};

// The tile of ticket t of group g (of the whole grid where there is no chain and so no counter).  Groups
// g = gb * nct + ct share out the blocks of channels and, in equal batches, the sequences gb, gb + gB, ...
// REV: later chunks of a sequence first.
template <bool REV> __device__ __forceinline__ Tile get_tile(const Seq &s, const Chunks &ch, uint32_t g, uint32_t t) {
    Tile o;
    o.ct = g % ch.nct;
    if (!s.off || ch.per == 1) {
        const int k = (int)(t / ch.nb);
        o.b = (int)(g / ch.nct + (t % ch.nb) * (ch.groups / ch.nct));
        o.k = REV ? ch.per - 1 - k : k;
        o.slot = (int64_t)o.b * ch.per + o.k;
        if (o.b >= s.B) o.b = 0, o.k = -1, o.slot = -1;
    } else {
        o.slot = REV ? ch.total - 1 - t : t;
        const Block k = packed_block(s, ch.tokens, o.slot);
        o.b = k.b;
        o.k = k.k;
    }
    return o;
}

template <bool CHAIN> __device__ __forceinline__ uint32_t take_ticket(const Chunks &ch, unsigned block, uint32_t g, uint32_t *shared) {
    if (!CHAIN) return block / ch.groups;
    if (threadIdx.x == 0) *shared = atomicAdd(ch.counter + g * kCounter, 1u);
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(*shared);
}

constexpr int kAhead = 2 * kWaves;      // maps read at once
template <int VEC> struct Links {
    float2 map[kAhead][64 * VEC];
    int found;
};

// The state that reaches a chunk from those at slot + dir, slot + 2 dir, ... (nearest first; `n` of them,
// the last of which publishes its state without waiting).  All waves of the workgroup: `leader` looks for
// the nearest published state; the maps between it and here, which may be as many as there are workgroups
// on the chip, are read by all waves at once, and folded by the leader, who gets h.
template <int VEC>
__device__ __forceinline__ void carry_in(const Chunks &ch, int C, int c, const Tile &tile, int dir, int n, bool leader,
                                         int w, Links<VEC> &sh, float (&h)[VEC]) {
    const int lane = threadIdx.x & 63;
    const int64_t step = (int64_t)dir * C;
    const uint32_t *sp = ch.state + tile.slot * C + c;
    const uint64_t *mp = ch.map + tile.slot * C + c;
    int polls = 0;
    if (leader) {
        int at = 1, found = 0;
        uint32_t u[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) u[v] = get(sp + step + v);      // most often it is the neighbour's
        while (!found) {
            const int i = at + lane;
            const uint32_t st = i <= n ? get(ch.stage + (tile.slot + (int64_t)dir * i) * ch.nct + tile.ct) : kNothing;
            const uint64_t states = __ballot(st == kState), some = __ballot(st != kNothing);
            const int lead = ~some ? __builtin_ctzll(~some) : 64;     // chunks in a row that have published something
            const int f = states ? __builtin_ctzll(states) : 64;
            if (f < lead) {
                found = at + f;
            } else if (lead == 64) {
                at += 64;
            } else {
                if (++polls > kMaxPolls) break;
                __builtin_amdgcn_s_sleep(1);
            }
        }
        bool ready = found == 1;
#pragma unroll
        for (int v = 0; v < VEC; ++v) ready = ready && u[v] != kEmpty;
        while (found && !__all(ready)) {
            ready = true;
#pragma unroll
            for (int v = 0; v < VEC; ++v) u[v] = get(sp + found * step + v);
#pragma unroll
            for (int v = 0; v < VEC; ++v) ready = ready && u[v] != kEmpty;
            if (++polls > kMaxPolls) found = 0;
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) h[v] = __uint_as_float(found ? u[v] : 0x7fc00000u);
        if (lane == 0) sh.found = found;
    }
    __syncthreads();
    for (int i = __builtin_amdgcn_readfirstlane(sh.found) - 1; i >= 1; i -= kAhead) {
        // wave w reads maps i - w, i - w - kWaves, ...
#pragma unroll
        for (int q = 0; q < kAhead / kWaves; ++q) {
            const int j = i - w - q * kWaves;
            if (j < 1) continue;
            uint64_t m[VEC];
            bool ok;
            do {
                ok = true;
#pragma unroll
                for (int v = 0; v < VEC; ++v) m[v] = get(mp + j * step + v);
#pragma unroll
                for (int v = 0; v < VEC; ++v) ok = ok && (uint32_t)m[v] != kEmpty;
            } while (!__all(ok) && ++polls <= kMaxPolls);
#pragma unroll
            for (int v = 0; v < VEC; ++v) sh.map[w + q * kWaves][lane * VEC + v] = make_float2(low(m[v]), high(m[v]));
        }
        __syncthreads();
        if (leader)
            for (int q = 0; q < min(i, kAhead); ++q)
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float2 m = sh.map[q][lane * VEC + v];
                    h[v] = fmaf(m.x, h[v], m.y);
                }
        __syncthreads();
    }
}

template <int VEC>
__device__ __forceinline__ void publish_map(const Chunks &ch, int C, int c, const Tile &t, const float (&A)[VEC],
                                            const float (&H)[VEC], bool on) {
    if (on) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) put(ch.map + t.slot * C + c + v, pair(A[v], H[v]));
    }
    put(ch.stage + t.slot * ch.nct + t.ct, (uint32_t)kMap);
}
template <int VEC>
__device__ __forceinline__ void publish_state(const Chunks &ch, int C, int c, const Tile &t, const float (&h)[VEC], bool on) {
    if (on) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) put(ch.state + t.slot * C + c + v, word(h[v]));
    }
    put(ch.stage + t.slot * ch.nct + t.ct, (uint32_t)kState);
}

// Empties the links (n units of 16 bytes of ones from ch.map on, zeros before), makes the channels'
// rates, and (block 0, packed sequences) the ascending offsets; the last workgroups fill rows of outputs.
__global__ __launch_bounds__(256) void scan_fill_kernel(Seq s, Chunks ch, int64_t n, float scale,
                                                        const float *__restrict__ decay, Fill f) {
    const unsigned links = gridDim.x - f.blocks;
    if (blockIdx.x >= links) {
        fill_rows(s, f, blockIdx.x - links, f.blocks);
        return;
    }
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) reinterpret_cast<uint4 *>(ch.map)[i] = make_uint4(kEmpty, kEmpty, kEmpty, kEmpty);
    if (i < ch.total * ch.nct) ch.stage[i] = kNothing;
    if (i < s.C) ch.rate[i] = scan_rate(scale, decay[i]);
    if (i < ch.groups) ch.counter[i * kCounter] = 0;
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

// The channels' rates, from the fill kernel or, where no sequence has a second chunk, made here.
template <int VEC, bool CHAIN>
__device__ __forceinline__ void get_rates(const Chunks &ch, float scale, const float *decay, int c, ScanRate (&k)[VEC]) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) k[v].set(CHAIN ? ch.rate[c + v] : scan_rate(scale, decay[c + v]));
}

// Lane addresses: a uniform row and a 32-bit byte offset, which the memory instructions add themselves.
template <typename T> __device__ __forceinline__ T *at_byte(T *row, uint32_t bytes) {
    return reinterpret_cast<T *>(const_cast<char *>(reinterpret_cast<const char *>(row)) + bytes);
}

// N rows from p on (uniform; off: this lane's channel, in bytes); only the first `there` of them exist, and the last
// of those stands in for the rest.
template <typename T, int VEC, int N, bool FULL, bool ONCE>
__device__ __forceinline__ void load_rows(typename Pack<T, VEC>::type (&v)[N], const T *p, int64_t ld, uint32_t off, int there) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = ONCE ? load_once<T, VEC>(at_byte(p, off)) : load_pack<T, VEC>(at_byte(p, off));
        if (FULL || i + 1 < there) p += ld;
    }
}

// Composed factors.  A product of many factors above 0 may underflow, and 0 * inf would then make NaN of an
// infinite state that each factor by itself passes on; so it stays at the smallest number there is, and is
// 0 only with a factor 0.  What that adds to a finite result is below 2^-149 of the state.
constexpr float kLeast = 0x1p-149f;
__device__ __forceinline__ float compose(float p, float q) {
    const float v = p * q;
    return v == 0.f && p != 0.f && q != 0.f ? kLeast : v;
}
// The same for the product A of a run's factors, which are looked at only where it is 0.
template <int VEC, int L> __device__ __forceinline__ void keep_positive(float (&A)[VEC], const float (&a)[L][VEC]) {
    bool under = false;
#pragma unroll
    for (int v = 0; v < VEC; ++v) under = under || A[v] == 0.f;
    if (!__any(under)) return;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        bool all = A[v] == 0.f;
#pragma unroll
        for (int i = 0; i < L; ++i) all = all && a[i][v] != 0.f;
        A[v] = all ? kLeast : A[v];
    }
}

// ---- forward -----------------------------------------------------------------------

// Tokens of a wave and of a workgroup.  Per lane 16 tokens of two channels: 48 loads under way, a and b in
// 64 registers, 119 in all, so two workgroups to a CU.  Four waves (71 us), 8 tokens (74 us) or
// one channel a lane (73 us) were slower than this (65 us at 8 x 2048 x 2048 bf16).
constexpr int kFwdRun = 16, kFwdChunk = kWaves * kFwdRun;

template <typename T, int VEC, bool CHAIN, bool ONCE>
__global__ __launch_bounds__(kThreads, 4) void scan_fwd_kernel(
    Seq s, float scale, const T *__restrict__ x, int64_t ldx, const T *__restrict__ gate, int64_t ldg,
    const T *__restrict__ inp, int64_t ldi, const float *__restrict__ decay, const float *__restrict__ h0,
    T *__restrict__ y, int64_t ldy, float *__restrict__ hT, float *__restrict__ states, Chunks ch, Fill f) {
    constexpr int L = kFwdRun, CW = 64 * VEC;
    __shared__ float sA[kWaves][CW], sH[kWaves][CW], sC[CW];
    __shared__ Links<VEC> sL;
    __shared__ uint32_t sTicket;
    unsigned block = blockIdx.x;
    if (!CHAIN) {                                  // the first workgroups fill; with chains the kernel in front of this one does
        if (block < (unsigned)f.blocks) {
            fill_rows(s, f, block, f.blocks);
            return;
        }
        block -= f.blocks;
    }
    const uint32_t group = block % ch.groups;
    const Tile tile = get_tile<false>(s, ch, group, take_ticket<CHAIN>(ch, block, group, &sTicket));
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
    const uint32_t off = (uint32_t)c * sizeof(T);
    const int tw = t0 + w * L, there = len - tw;   // this wave's tokens: L from tw on, or `there`
    float a[L][VEC], bb[L][VEC], A[VEC], H[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) A[v] = 1.f, H[v] = 0.f;
    const auto read = [&](auto full_) {
        constexpr bool full = decltype(full_)::value;
        typename Pack<T, VEC>::type xr[L], gr[L], ir[L];
        load_rows<T, VEC, L, full, ONCE>(gr, gate + (first + tw) * ldg, ldg, off, there);
        load_rows<T, VEC, L, full, ONCE>(ir, inp + (first + tw) * ldi, ldi, off, there);
        load_rows<T, VEC, L, full, ONCE>(xr, x + (first + tw) * ldx, ldx, off, there);
        ScanRate k[VEC];
        get_rates<VEC, CHAIN>(ch, scale, decay, c, k);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            float xv[VEC], gv[VEC], iv[VEC];
            to_f32(xr[i], xv);
            to_f32(gr[i], gv);
            to_f32(ir[i], iv);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const ScanGates g(k[v], gv[v], iv[v]);
                a[i][v] = full || i < there ? g.a : 1.f;
                bb[i][v] = full || i < there ? g.m * g.s * xv[v] : 0.f;
                A[v] *= a[i][v];
                H[v] = fmaf(a[i][v], H[v], bb[i][v]);
            }
        }
        keep_positive(A, a);
    };
    if (there >= L)
        read(std::true_type{});
    else if (there > 0)
        read(std::false_type{});
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
            PA[v] = compose(PA[v], Aq);
        }
    float c0[VEC];
    const bool more = CHAIN && t0 + kFwdChunk < len;
    if (w == kWaves - 1) {                       // this wave has the whole chunk's map
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            H[v] = fmaf(A[v], PH[v], H[v]);
            A[v] = compose(A[v], PA[v]);
        }
        if (tile.k == 0) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) c0[v] = h0 ? h0[(int64_t)b * C + c + v] : 0.f;
        } else if (CHAIN) {
            if (more) publish_map<VEC>(ch, C, c, tile, A, H, on);
        }
    }
    if (CHAIN && tile.k > 0) carry_in<VEC>(ch, C, c, tile, -1, tile.k, w == kWaves - 1, w, sL, c0);
    if (w == kWaves - 1) {
        float out[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) out[v] = fmaf(A[v], c0[v], H[v]);
        if (more) publish_state<VEC>(ch, C, c, tile, out, on);
#pragma unroll
        for (int v = 0; v < VEC; ++v) sC[lane * VEC + v] = c0[v];
    }
    __syncthreads();
    float h[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = fmaf(PA[v], sC[lane * VEC + v], PH[v]);
    if (!on) return;
    if (states && there > 0 && tw % kBlock == 0) {
        const int64_t nb = (s.T + kBlock - 1) / kBlock;
#pragma unroll
        for (int v = 0; v < VEC; ++v) states[(b * nb + tw / kBlock) * C + c + v] = h[v];
    }
    const auto write = [&](auto full_) {
        constexpr bool full = decltype(full_)::value;
        T *yp = y + (first + tw) * ldy;
#pragma unroll
        for (int i = 0; i < L; ++i) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) h[v] = fmaf(a[i][v], h[v], bb[i][v]);
            if (full || i < there) store_f32<ONCE>(at_byte(yp, off), h);
            yp += ldy;
        }
    };
    if (there >= L)
        write(std::true_type{});
    else if (there > 0)
        write(std::false_type{});
    // the wave of the last token, or of an empty sequence the first one
    if (hT && (there > 0 ? there <= L : len == 0 && w == 0))
#pragma unroll
        for (int v = 0; v < VEC; ++v) hT[(int64_t)b * C + c + v] = h[v];
}

// ---- backward ----------------------------------------------------------------------
//
// e[t] = a[t] dh[t] is what the gradient of h[t-1] receives: e_in -> a (dy + e_in)
// is affine with the same factor, so the chunks chain as in the forward pass, the
// other way round.  h[t-1] is run forward again from the saved state at the
// chunk's start, in the same pass over the registers: reading y instead would cost
// 2 bytes more an element and bring its rounding into the gradients.  dk leaves one
// partial sum per chunk and channel, added in order by scan_reduce_kernel.  Runs of
// 8 tokens: what has to be kept of each (five values, x and dy) fills 128 registers.

constexpr int kBwdRun = 8, kBwdChunk = kWaves * kBwdRun;
static_assert(kBwdChunk == kBlock, "a saved state for every chunk");

template <typename T, int VEC, bool CHAIN, bool ONCE>
__global__ __launch_bounds__(kThreads, 4) void scan_bwd_kernel(
    Seq s, float scale, const T *__restrict__ x, int64_t ldx, const T *__restrict__ gate, int64_t ldg,
    const T *__restrict__ inp, int64_t ldi, const float *__restrict__ decay, const float *__restrict__ states,
    const T *__restrict__ dy, int64_t lddy, const float *__restrict__ dhT, T *__restrict__ dx, int64_t lddx,
    T *__restrict__ dgate, int64_t lddg, T *__restrict__ dinp, int64_t lddi, float *__restrict__ part,
    float *__restrict__ dh0, Chunks ch, Fill f) {
    constexpr int L = kBwdRun, CW = 64 * VEC;
    __shared__ float sA[kWaves][CW], sH[kWaves][CW], sE[kWaves][CW], sC[CW];
    __shared__ Links<VEC> sL;
    __shared__ uint32_t sTicket;
    unsigned block = blockIdx.x;
    if (!CHAIN) {                                  // the first workgroups fill; with chains the kernel in front of this one does
        if (block < (unsigned)f.blocks) {
            fill_rows(s, f, block, f.blocks);
            return;
        }
        block -= f.blocks;
    }
    const uint32_t group = block % ch.groups;
    const Tile tile = get_tile<true>(s, ch, group, take_ticket<CHAIN>(ch, block, group, &sTicket));
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int b = tile.b, C = s.C;
    int64_t first;
    int len;
    seq_range(s, b, first, len);
    const int t0 = tile.k * kBwdChunk;
    const int cw = tile.ct * CW + lane * VEC;
    const bool on = cw < C;
    const int c = min(cw, C - VEC);                // odd C: the last lane shares a channel, with the same results
    const uint32_t off = (uint32_t)c * sizeof(T);
    if (tile.slot < 0) return;                     // no sequence
    if (tile.k < 0 || t0 >= len) {                 // an unused number, or an empty sequence
        if (on && w == 0)
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                part[tile.slot * C + c + v] = 0.f;
                if (len == 0 && tile.k == 0 && dh0)
                    dh0[(int64_t)b * C + c + v] = dhT ? dhT[(int64_t)b * C + c + v] : 0.f;
            }
        return;
    }
    const int tw = t0 + w * L, there = len - tw;
    float h[VEC], A[VEC], H[VEC], E[VEC];
    // per token: a, r, s; ms = m s; and q = s x a / m, later a (h[t-1] - q)
    float a[L][VEC], r[L][VEC], sg[L][VEC], ms[L][VEC], q[L][VEC];
    typename Pack<T, VEC>::type xr[L], dr[L];
    ScanRate k[VEC];
    const int64_t nb = (s.T + kBlock - 1) / kBlock;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        A[v] = 1.f, H[v] = 0.f, E[v] = 0.f;
        h[v] = states[(b * nb + tile.k) * C + c + v];
    }
    const auto read = [&](auto full_) {
        constexpr bool full = decltype(full_)::value;
        typename Pack<T, VEC>::type gr[L], ir[L];
        load_rows<T, VEC, L, full, ONCE>(gr, gate + (first + tw) * ldg, ldg, off, there);
        load_rows<T, VEC, L, full, ONCE>(ir, inp + (first + tw) * ldi, ldi, off, there);
        load_rows<T, VEC, L, full, ONCE>(xr, x + (first + tw) * ldx, ldx, off, there);
        load_rows<T, VEC, L, full, ONCE>(dr, dy + (first + tw) * lddy, lddy, off, there);
        get_rates<VEC, CHAIN>(ch, scale, decay, c, k);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            float xv[VEC], gv[VEC], iv[VEC];
            to_f32(xr[i], xv);
            to_f32(gr[i], gv);
            to_f32(ir[i], iv);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const ScanGates g(k[v], gv[v], iv[v]);
                const bool in = full || i < there;
                a[i][v] = in ? g.a : 1.f;
                r[i][v] = g.r, sg[i][v] = g.s, ms[i][v] = in ? g.m * g.s : 0.f;
                q[i][v] = g.s * xv[v] * g.a * g.im;
                A[v] *= a[i][v];
                H[v] = fmaf(a[i][v], H[v], ms[i][v] * xv[v]);
            }
        }
        keep_positive(A, a);
#pragma unroll
        for (int i = L - 1; i >= 0; --i) {
            float dv[VEC];
            to_f32(dr[i], dv);
#pragma unroll
            for (int v = 0; v < VEC; ++v) E[v] = a[i][v] * (full || i < there ? dv[v] + E[v] : E[v]);
        }
    };
    if (there >= L)
        read(std::true_type{});
    else if (there > 0)
        read(std::false_type{});
#pragma unroll
    for (int v = 0; v < VEC; ++v)
        sA[w][lane * VEC + v] = A[v], sH[w][lane * VEC + v] = H[v], sE[w][lane * VEC + v] = E[v];
    __syncthreads();
    // h in front of this wave's tokens; the map from the chunk's e_in to this wave's
    float PA[VEC], PE[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) PA[v] = 1.f, PE[v] = 0.f;
    for (int p = 0; p < w; ++p)
#pragma unroll
        for (int v = 0; v < VEC; ++v) h[v] = fmaf(sA[p][lane * VEC + v], h[v], sH[p][lane * VEC + v]);
    for (int p = kWaves - 1; p > w; --p)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float Aq = sA[p][lane * VEC + v];
            PE[v] = fmaf(Aq, PE[v], sE[p][lane * VEC + v]);
            PA[v] = compose(PA[v], Aq);
        }
    float c0[VEC];
    const int behind = (len + kBwdChunk - 1) / kBwdChunk - 1 - tile.k;           // chunks after this one
    const bool more = CHAIN && tile.k > 0;
    if (w == 0) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            E[v] = fmaf(A[v], PE[v], E[v]);
            A[v] = compose(A[v], PA[v]);
        }
        if (!CHAIN || behind == 0) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) c0[v] = dhT ? dhT[(int64_t)b * C + c + v] : 0.f;
        } else {
            if (more) publish_map<VEC>(ch, C, c, tile, A, E, on);
        }
    }
    // h forward through this wave's tokens
#pragma unroll
    for (int i = 0; i < L; ++i) {
        if (i < there) {
            float xv[VEC];
            to_f32(xr[i], xv);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                q[i][v] = a[i][v] * (h[v] - q[i][v]);
                h[v] = fmaf(a[i][v], h[v], ms[i][v] * xv[v]);
            }
        }
    }
    if (CHAIN && behind > 0) carry_in<VEC>(ch, C, c, tile, 1, behind, w == 0, w, sL, c0);
    if (w == 0) {
        float out[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) out[v] = fmaf(A[v], c0[v], E[v]);
        if (more) publish_state<VEC>(ch, C, c, tile, out, on);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            if (on && dh0 && tile.k == 0) dh0[(int64_t)b * C + c + v] = out[v];
            sC[lane * VEC + v] = c0[v];
        }
    }
    __syncthreads();
    float dk[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) dk[v] = 0.f;
    const auto write = [&](auto full_) {
        constexpr bool full = decltype(full_)::value;
        float e[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) e[v] = fmaf(PA[v], sC[lane * VEC + v], PE[v]);
        const int last = full ? L - 1 : there - 1;
        T *dxp = dx + (first + tw + last) * lddx, *dgp = dgate + (first + tw + last) * lddg,
          *dip = dinp + (first + tw + last) * lddi;
#pragma unroll
        for (int i = L - 1; i >= 0; --i) {
            if (!full && i >= there) continue;
            float xv[VEC], dv[VEC], o0[VEC], o1[VEC], o2[VEC];
            to_f32(xr[i], xv);
            to_f32(dr[i], dv);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float dh = dv[v] + e[v], rdla = r[i][v] * (dh * q[i][v]);
                o0[v] = dh * ms[i][v];
                o1[v] = -k[v].k * rdla * (1.f - r[i][v]);
                o2[v] = o0[v] * xv[v] * (1.f - sg[i][v]);
                dk[v] += rdla;
                e[v] = a[i][v] * dh;
            }
            if (on) {
                store_f32<ONCE>(at_byte(dxp, off), o0);
                store_f32<ONCE>(at_byte(dgp, off), o1);
                store_f32<ONCE>(at_byte(dip, off), o2);
            }
            dxp -= lddx;
            dgp -= lddg;
            dip -= lddi;
        }
    };
    if (there >= L)
        write(std::true_type{});
    else if (there > 0)
        write(std::false_type{});
    // sA is free: every wave read it before the barrier above
#pragma unroll
    for (int v = 0; v < VEC; ++v) sA[w][lane * VEC + v] = dk[v];
    __syncthreads();
    if (w == 0 && on)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            float d = 0.f;
            for (int p = 0; p < kWaves; ++p) d += sA[p][lane * VEC + v];
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
    ScanRate k;
    k.set(scan_rate(scale, decay[c]));
    const ScanGates g(k, gv[0], iv[0]);
    const float o[1] = {fmaf(g.a, h[i], g.m * g.s * xv[0])};
    h[i] = o[0];
    store_f32(y + b * ldy + c, o);
}

Chunks chunks(const Seq &s, int tokens) {
    Chunks ch = {};
    ch.tokens = tokens;
    ch.per = s.T > 0 ? (s.T + tokens - 1) / tokens : 1;
    ch.nct = (s.C + 63) / 64;          // of the narrowest kernel: the workspace does not depend on the dtype
    ch.total = block_count(s, tokens, ch.per);
    return ch;
}

// Groups for `channels` channels a workgroup; returns the workgroups there are.
int64_t set_groups(const Seq &s, Chunks &ch, int channels) {
    ch.nct = (s.C + channels - 1) / channels;
    const ScanGrid g = scan_grid(s.B, ch.nct, ch.per, s.off && ch.per > 1 ? ch.total : 0);
    ch.groups = g.groups;
    ch.nb = g.nb;
    return g.size;
}

// Workspace of the links: the counter, the offsets, the rates, the stages, and then per chunk and channel
// 8 bytes of map and 4 of state, each part to a multiple of 16; none if no sequence has a second chunk.
int64_t counter_bytes(const Chunks &ch) { return 4 * kCounter * (int64_t)std::max(64, ch.nct); }
int64_t pad16(int64_t bytes) { return (bytes + 15) / 16 * 16; }
int64_t off_bytes(const Seq &s) { return s.off ? pad16(4 * ((int64_t)s.B + 1)) : 0; }
int64_t stage_bytes(const Chunks &ch) { return pad16(4 * ch.total * ch.nct); }
int64_t link_units(const Seq &s, const Chunks &ch) { return pad16(ch.total * s.C * 12) / 16; }
size_t link_bytes(const Seq &s, const Chunks &ch) {
    return ch.per > 1 ? (size_t)(counter_bytes(ch) + off_bytes(s) + pad16(4 * s.C) + stage_bytes(ch) + 16 * link_units(s, ch)) : 0;
}

// Lays the links out in ws and empties them; s then has the ascending offsets.  grid: workgroups.
// f: the rows to fill; where there is no second chunk, and so no kernel for the links, the main one fills them
// with workgroups of its own, if its grid has room for them.
hipError_t set_links(Seq &s, Chunks &ch, void *ws, int channels, float scale, const float *decay, int64_t &grid, Fill &f,
                     hipStream_t st) {
    char *p = (char *)ws;
    const Chunks sizes = ch;
    grid = set_groups(s, ch, channels);
    if (ch.per <= 1) {
        if (f.blocks) f.blocks = (int)std::min<int64_t>(f.blocks, kScanMaxGrid - grid);
        grid += f.blocks;
        return hipSuccess;
    }
    ch.counter = (uint32_t *)p;
    ch.off = (int32_t *)(p += counter_bytes(sizes));
    ch.rate = (float *)(p += off_bytes(s));
    ch.stage = (uint32_t *)(p += pad16(4 * s.C));
    ch.map = (uint64_t *)(p += stage_bytes(sizes));
    ch.state = (uint32_t *)(ch.map + ch.total * s.C);
    // one thread per unit of the links, per stage, per channel and per counter
    const int64_t n = link_units(s, ch), threads = std::max({n, ch.total * ch.nct, (int64_t)s.C, (int64_t)ch.groups});
    scan_fill_kernel<<<(unsigned)((threads + 255) / 256) + f.blocks, 256, 0, st>>>(s, ch, n, scale, decay, f);
    if (s.off) s.off = ch.off;
    return hipGetLastError();
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
                     Chunks ch, int64_t grid, const Fill &f, hipStream_t st) {
    const bool once = read_once(x, ldx, sizeof(T)) && read_once(gate, ldg, sizeof(T)) && read_once(inp, ldi, sizeof(T)) &&
                      read_once(y, ldy, sizeof(T));
    const auto run = ch.per > 1 ? (once ? scan_fwd_kernel<T, VEC, true, true> : scan_fwd_kernel<T, VEC, true, false>)
                                : (once ? scan_fwd_kernel<T, VEC, false, true> : scan_fwd_kernel<T, VEC, false, false>);
    run<<<(unsigned)grid, kThreads, 0, st>>>(s, scale, (const T *)x, ldx, (const T *)gate, ldg, (const T *)inp, ldi,
                                                         decay, h0, (T *)y, ldy, hT, states, ch, f);
}

hipError_t launch_scan_fwd(const Seq &s, bool bf16, float scale, const void *x, int64_t ldx, const void *gate,
                           int64_t ldg, const void *inp, int64_t ldi, const float *decay, const float *h0, void *y,
                           int64_t ldy, float *hT, float *states, void *ws, hipStream_t st) {
    Chunks ch = chunks(s, kFwdChunk);
    Seq q = s;
    int64_t grid;
    const int waves = ch.per > 1 ? 4 : kWaves;
    Fill f = bf16 ? fill_of<uint16_t>(s, waves, {(uint16_t *)y}, {ldy}) : fill_of<float>(s, waves, {(float *)y}, {ldy});
    const hipError_t e = set_links(q, ch, ws, bf16 && s.C > 1 ? 128 : 64, scale, decay, grid, f, st);
    if (e != hipSuccess) return e;              // no chunk may be taken from counters that are not set
    const auto run = !bf16 ? scan_fwd<float, 1> : s.C > 1 ? scan_fwd<uint16_t, 2> : scan_fwd<uint16_t, 1>;
    run(q, scale, x, ldx, gate, ldg, inp, ldi, decay, h0, y, ldy, hT, states, ch, grid, f, st);
    return hipGetLastError();
}

template <typename T, int VEC>
static void scan_bwd(const Seq &s, float scale, const void *x, int64_t ldx, const void *gate, int64_t ldg, const void *inp,
                     int64_t ldi, const float *decay, const float *states, const void *dy, int64_t lddy, const float *dhT,
                     void *dx, int64_t lddx, void *dgate, int64_t lddg, void *dinp, int64_t lddi, float *part, float *dh0,
                     Chunks ch, int64_t grid, const Fill &f, hipStream_t st) {
    const bool once = read_once(x, ldx, sizeof(T)) && read_once(gate, ldg, sizeof(T)) && read_once(inp, ldi, sizeof(T)) &&
                      read_once(dy, lddy, sizeof(T)) && read_once(dx, lddx, sizeof(T)) && read_once(dgate, lddg, sizeof(T)) &&
                      read_once(dinp, lddi, sizeof(T));
    const auto run = ch.per > 1 ? (once ? scan_bwd_kernel<T, VEC, true, true> : scan_bwd_kernel<T, VEC, true, false>)
                                : (once ? scan_bwd_kernel<T, VEC, false, true> : scan_bwd_kernel<T, VEC, false, false>);
    run<<<(unsigned)grid, kThreads, 0, st>>>(s, scale, (const T *)x, ldx, (const T *)gate, ldg, (const T *)inp, ldi,
                                                         decay, states, (const T *)dy, lddy, dhT, (T *)dx, lddx, (T *)dgate,
                                                         lddg, (T *)dinp, lddi, part, dh0, ch, f);
}

hipError_t launch_scan_bwd(const Seq &s, bool bf16, float scale, const void *x, int64_t ldx, const void *gate, int64_t ldg,
                           const void *inp, int64_t ldi, const float *decay, const float *states, const void *dy, int64_t lddy,
                           const float *dhT, void *dx, int64_t lddx, void *dgate, int64_t lddg, void *dinp, int64_t lddi,
                           float *ddecay, float *dh0, void *ws, hipStream_t st) {
    Chunks ch = chunks(s, kBwdChunk);
    Seq q = s;
    int64_t grid;
    const int waves = ch.per > 1 ? 4 : kWaves;
    const std::initializer_list<int64_t> lds = {lddx, lddg, lddi};
    Fill f = bf16 ? fill_of<uint16_t>(s, waves, {(uint16_t *)dx, (uint16_t *)dgate, (uint16_t *)dinp}, lds)
                  : fill_of<float>(s, waves, {(float *)dx, (float *)dgate, (float *)dinp}, lds);
    const hipError_t e = set_links(q, ch, ws, bf16 && s.C > 1 ? 128 : 64, scale, decay, grid, f, st);
    if (e != hipSuccess) return e;              // no chunk may be taken from counters that are not set
    float *part = (float *)((char *)ws + link_bytes(s, chunks(s, kBwdChunk)));
    const auto run = !bf16 ? scan_bwd<float, 1> : s.C > 1 ? scan_bwd<uint16_t, 2> : scan_bwd<uint16_t, 1>;
    run(q, scale, x, ldx, gate, ldg, inp, ldi, decay, states, dy, lddy, dhT, dx, lddx, dgate, lddg, dinp, lddi, part, dh0, ch,
        grid, f, st);
    const hipError_t e2 = hipGetLastError();
    if (e2 != hipSuccess) return e2;            // there are no partial sums
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
