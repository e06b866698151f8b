// scan_grid.h -- how many workgroups the recurrence takes and how they share
// out the chunks.  Host arithmetic only.
#pragma once

#include <stdint.h>

namespace convfwd {

constexpr int kScanThreads = 512;
constexpr int64_t kScanMaxGrid = (INT64_C(1) << 32) / kScanThreads - 1;    // a launch counts its threads in 32 bits

// Some 64 groups of workgroups, each with a counter: all nct blocks of channels, times as many batches of
// sequences.  Sequences gb, gb + gB, ... belong to batch gb of gB; nb: sequences of a batch (the last places
// may be empty).
struct ScanGrid {
    int groups, nb;
    int64_t size;
};

// B sequences of `per` chunks each; through > 0: chunks are numbered through, `through` of them, and stay together.
inline ScanGrid scan_grid(int B, int nct, int per, int64_t through) {
    if (through > 0) return ScanGrid{nct, B, nct * through};
    const int64_t tiles = (int64_t)nct * per;
    int gB = nct >= 64 ? 1 : 64 / nct;
    if (gB > B) gB = B;
    ScanGrid g;
    g.nb = (B + gB - 1) / gB;
    // Where the empty places of the last batches are too many for a launch: no more batches than nb sequences each
    // need (65 sequences make 33 of two, not 64), or one batch, which has none.  Otherwise more counters are better
    // (65 x 512 x 512 forward: 40.1 us with 16 batches of five, 41.3 with 13).
    if (tiles * gB * g.nb >= kScanMaxGrid) gB = (B + g.nb - 1) / g.nb;
    if (tiles * gB * g.nb >= kScanMaxGrid) gB = 1, g.nb = B;
    g.groups = nct * gB;
    g.size = tiles * gB * g.nb;
    return g;
}

}  // namespace convfwd
