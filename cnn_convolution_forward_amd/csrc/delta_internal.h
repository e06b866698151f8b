// delta_internal.h -- launchers of the gated delta rule (k_delta*.hip).  Each
// enqueues on `st` and returns hipGetLastError(); arguments have been checked
// (delta_api.cpp).
#pragma once

#include "seq_internal.h"

namespace convfwd {

// conv_delta_t as the kernels see it.
struct Delta {
    int H, Hv, Dk, Dv, group;      // group = Hv / H value heads share a query and key head
    bool unit;
    float scale, eps;
};

// Rows of one tensor and the elements between them.
struct Rows {
    const void *p;
    int64_t ld;
};
struct RowsOut {
    void *p;
    int64_t ld;
};
struct DeltaIn {
    Rows q, k, v, g, beta;         // g and beta are fp32
};

size_t delta_fwd_workspace(const Seq &s, const Delta &d, bool bf16);      // bytes
hipError_t launch_delta_fwd(const Seq &s, const Delta &d, bool bf16, const DeltaIn &in, const float *s0, RowsOut y, float *sT,
                            float *states, void *ws, hipStream_t st);
size_t delta_bwd_workspace(const Seq &s, const Delta &d, bool bf16);
hipError_t launch_delta_bwd(const Seq &s, const Delta &d, bool bf16, const DeltaIn &in, const float *states, Rows dy, const float *dsT,
                            RowsOut dq, RowsOut dk, RowsOut dv, RowsOut dg, RowsOut dbeta, float *ds0, void *ws, hipStream_t st);
hipError_t launch_delta_step(const Seq &s, const Delta &d, bool bf16, const DeltaIn &in, float *S, RowsOut y, hipStream_t st);

}  // namespace convfwd
