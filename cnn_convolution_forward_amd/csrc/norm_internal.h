// norm_internal.h -- launchers of the layer norm (k_norm.hip).  Each enqueues
// on `st` and returns hipGetLastError(); arguments have been checked
// (seq_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace convfwd {

hipError_t launch_norm_fwd(int64_t rows, int C, bool bf16, float eps, const void *x, int64_t ldx, const float *w, const float *b,
                           void *y, int64_t ldy, float *mean, float *rstd, hipStream_t st);
int64_t norm_bwd_workspace_floats(int64_t rows, int C, bool bf16);
// part: norm_bwd_workspace_floats floats (may be NULL where neither dw nor db is wanted)
hipError_t launch_norm_bwd(int64_t rows, int C, bool bf16, const void *x, int64_t ldx, const float *w, const float *mean,
                           const float *rstd, const void *dy, int64_t lddy, void *dx, int64_t lddx, float *dw, float *db,
                           float *part, hipStream_t st);

}  // namespace convfwd
