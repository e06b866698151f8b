// seq_internal.h -- launchers of the operators over sequences of tokens
// (k_seqconv.hip, k_scan.hip).  Each enqueues on `st` and returns
// hipGetLastError(); arguments have been checked (seq_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace convfwd {

// conv_seq_t as the kernels see it.
struct Seq {
    int B, T, C;
    const int32_t *off;      // NULL: sequence b is rows [b*T, (b+1)*T)
    int64_t rows;            // rows of x: B*T, or the packed tensor's
    bool fill;               // packed: rows of outputs that no sequence holds become zero
};

int64_t causal_bwd_workspace_floats(const Seq &s, int K);
hipError_t launch_causal_fwd(const Seq &s, bool bf16, int K, int silu, const void *x, int64_t ldx, const void *w,
                             const float *bias, const void *state, void *y, int64_t ldy, void *state_out, hipStream_t st);
// part: causal_bwd_workspace_floats floats
hipError_t launch_causal_bwd(const Seq &s, bool bf16, int K, int silu, const void *x, int64_t ldx, const void *w,
                             const float *bias, const void *state, const void *dy, int64_t lddy, void *dx, int64_t lddx,
                             float *dw, float *db, void *dstate, float *part, hipStream_t st);
hipError_t launch_causal_step(const Seq &s, bool bf16, int K, int silu, const void *x, int64_t ldx, const void *w,
                              const float *bias, void *state, void *y, int64_t ldy, hipStream_t st);

size_t scan_fwd_workspace(const Seq &s);      // bytes
size_t scan_bwd_workspace(const Seq &s);
hipError_t launch_scan_fwd(const Seq &s, bool bf16, float scale, const void *x, int64_t ldx, const void *gate,
                           int64_t ldg, const void *inp, int64_t ldi, const float *decay, const float *h0, void *y,
                           int64_t ldy, float *hT, float *states, void *ws, hipStream_t st);
hipError_t launch_scan_bwd(const Seq &s, bool bf16, float scale, const void *x, int64_t ldx, const void *gate,
                           int64_t ldg, const void *inp, int64_t ldi, const float *decay, const float *states,
                           const void *dy, int64_t lddy, const float *dhT, void *dx, int64_t lddx, void *dgate,
                           int64_t lddg, void *dinp, int64_t lddi, float *ddecay, float *dh0, void *ws, hipStream_t st);
hipError_t launch_scan_step(const Seq &s, bool bf16, float scale, const void *x, int64_t ldx, const void *gate,
                            int64_t ldg, const void *inp, int64_t ldi, const float *decay, float *h, void *y,
                            int64_t ldy, hipStream_t st);

}  // namespace convfwd
