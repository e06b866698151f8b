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
    ScanGrid g;
    int gB = nct >= 64 ? 1 : 64 / nct;
    if (gB > B) gB = B;
    g.nb = (B + gB - 1) / gB;
    gB = (B + g.nb - 1) / g.nb;              // no more batches than nb sequences each need: 65 make 33 batches of two, not 64
    if ((int64_t)nct * per * gB * g.nb > kScanMaxGrid) gB = 1, g.nb = B;      // no empty places at all
    g.groups = nct * gB;
    g.size = (int64_t)g.groups * per * g.nb;
    return g;
}

}  // namespace convfwd
