// seq_checks.h -- what the entry points over sequences of tokens check of their
// arguments, on the host and before any HIP call (seq_api.cpp, delta_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "conv_fwd.h"
#include "seq_internal.h"

namespace convfwd {

constexpr int64_t kMaxRows = INT64_C(1) << 30;
constexpr int64_t kMaxBlocks = INT64_C(1) << 23;       // 64-token blocks of all sequences, and these times
                                                       // 64-channel blocks: grid dimensions
constexpr int kMaxChannels = 1 << 20;
constexpr int64_t kMaxStateElems = INT64_C(2147483647);

inline conv_status_t to_status(hipError_t e) { return e == hipSuccess ? CONV_OK : CONV_ERR_HIP; }

// One operand: `rows` rows of `cols` elements of `esize` bytes, `ld` elements apart.
struct Span {
    const void *p;
    int64_t rows, cols, ld;
    int esize;
    bool empty() const { return !p || rows <= 0 || cols <= 0; }
    uintptr_t begin() const { return (uintptr_t)p; }
    uintptr_t end() const { return begin() + (uintptr_t)(((rows - 1) * ld + cols) * esize); }
};

inline Span dense(const void *p, int64_t elems, int esize) { return Span{p, 1, elems, elems, esize}; }

inline bool overlap(const Span &a, const Span &b) {
    if (a.empty() || b.empty() || a.begin() >= b.end() || b.begin() >= a.end()) return false;
    // Column slices of one buffer: the same distance between rows, and columns that do not meet
    // within it.
    const int64_t step = a.ld * a.esize;
    if (a.rows > 1 && b.rows > 1 && step == b.ld * b.esize) {
        int64_t d = (int64_t)(b.begin() - a.begin()) % step;
        if (d < 0) d += step;
        return d < a.cols * a.esize || d + b.cols * b.esize > step;
    }
    return true;
}

inline conv_status_t check_alias(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span *o = outs.begin(); o != outs.end(); ++o) {
        for (const Span &i : ins)
            if (overlap(*o, i)) return CONV_ERR_ALIAS;
        for (const Span *q = o + 1; q != outs.end(); ++q)
            if (overlap(*o, *q)) return CONV_ERR_ALIAS;
    }
    return CONV_OK;
}

inline conv_status_t check_align(std::initializer_list<Span> all) {
    for (const Span &s : all)
        if ((uintptr_t)s.p % s.esize || (s.rows > 0 && s.ld < s.cols)) return CONV_ERR_PARAM;
    return CONV_OK;
}

// step: one row for each sequence.
inline conv_status_t make_seq(const conv_seq_t *q, bool step, Seq &s) {
    if (!q) return CONV_ERR_NULL;
    const int dtype = q->dtype & ~CONV_SEQ_FILL;
    if ((dtype != CONV_OUT_F32 && dtype != CONV_OUT_BF16) || q->B < 1 || q->C < 1) return CONV_ERR_PARAM;
    if (!step && (q->T < 0 || (q->offsets && q->tokens < 0) || (uintptr_t)q->offsets % 4)) return CONV_ERR_PARAM;
    s.B = q->B;
    s.C = q->C;
    s.T = step ? 1 : q->T;
    s.off = step ? nullptr : q->offsets;
    s.rows = s.off ? q->tokens : (int64_t)s.B * s.T;
    s.fill = s.off && (q->dtype & CONV_SEQ_FILL);
    if (s.rows >= kMaxRows || s.T >= kMaxRows || s.C > kMaxChannels || (int64_t)s.B * s.C > kMaxStateElems ||
        s.rows / CONV_SCAN_BLOCK + 2 * (int64_t)s.B > kMaxBlocks ||
        (s.rows / CONV_SCAN_BLOCK + s.B) * ((s.C + 63) / 64) > kMaxBlocks)
        return CONV_ERR_OVERFLOW;
    return CONV_OK;
}

inline int esize(const conv_seq_t *q) { return (q->dtype & ~CONV_SEQ_FILL) == CONV_OUT_BF16 ? 2 : 4; }

inline conv_status_t check_workspace(const void *ws, size_t bytes, size_t need) {
    return need && (!ws || bytes < need || (uintptr_t)ws % 16) ? CONV_ERR_WORKSPACE : CONV_OK;
}

}  // namespace convfwd

#define TRY(e)                                   \
    do {                                         \
        const conv_status_t st_ = (e);           \
        if (st_ != CONV_OK) return st_;          \
    } while (0)
