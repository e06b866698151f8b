// delta_api.cpp -- the extern "C" entry points of the gated delta rule.  As in
// seq_api.cpp, every argument is checked on the host before any HIP call.
#include <math.h>

#include "delta_internal.h"
#include "seq_checks.h"

using namespace convfwd;

namespace {

constexpr int kMaxDim = 128;
constexpr int64_t kMaxHeadBlocks = INT64_C(1) << 21;
constexpr int64_t kMaxStep = INT64_C(1) << 22;         // elements between rows: a block's rows stay below 2^30 bytes

conv_status_t make_delta(const conv_seq_t *q, const conv_delta_t *p, bool step, Seq &s, Delta &d) {
    if (!p) return CONV_ERR_NULL;
    TRY(make_seq(q, step, s));
    if (p->heads < 1 || p->heads_v < 1 || p->heads_v % p->heads || p->dim_k < 1 || p->dim_k > kMaxDim || p->dim_v < 1 ||
        p->dim_v > kMaxDim || (int64_t)p->heads_v * p->dim_v != s.C || (p->unit != 0 && p->unit != 1) || !isfinite(p->scale) ||
        !(p->eps >= 0.f) || isinf(p->eps))
        return CONV_ERR_PARAM;
    if ((int64_t)s.B * p->heads_v * p->dim_k * p->dim_v > kMaxStateElems || (s.rows / 64 + s.B) * p->heads_v >= kMaxHeadBlocks)
        return CONV_ERR_OVERFLOW;
    d.H = p->heads, d.Hv = p->heads_v, d.Dk = p->dim_k, d.Dv = p->dim_v, d.group = p->heads_v / p->heads;
    d.unit = p->unit != 0;
    d.scale = p->scale, d.eps = p->eps;
    return CONV_OK;
}

// The spans of the inputs of n rows.
struct Inputs {
    Span q, k, v, g, b;
};
Inputs inputs(const DeltaIn &in, const Delta &d, int64_t n, int e) {
    const auto rows = [n](const Rows &r, int64_t cols, int esize) { return Span{r.p, n, cols, r.ld, esize}; };
    return {rows(in.q, (int64_t)d.H * d.Dk, e), rows(in.k, (int64_t)d.H * d.Dk, e), rows(in.v, (int64_t)d.Hv * d.Dv, e),
            rows(in.g, d.Hv, 4), rows(in.beta, d.Hv, 4)};
}

conv_status_t check_steps(std::initializer_list<Span> all) {
    for (const Span &s : all)
        if (s.ld >= kMaxStep) return CONV_ERR_OVERFLOW;
    return CONV_OK;
}

}  // namespace

extern "C" {

size_t conv_delta_fwd_workspace_bytes(const conv_seq_t *seq, const conv_delta_t *par) {
    Seq s;
    Delta d;
    return make_delta(seq, par, false, s, d) == CONV_OK ? delta_fwd_workspace(s, d, esize(seq) == 2) : 0;
}

conv_status_t conv_delta_fwd(const conv_seq_t *seq, const conv_delta_t *par, const void *q, int64_t ldq, const void *k,
                             int64_t ldk, const void *v, int64_t ldv, const float *gate, int64_t ldg, const float *beta,
                             int64_t ldb, const float *s0, void *y, int64_t ldy, float *sT, float *states, void *workspace,
                             size_t workspace_bytes, void *stream) {
    Seq s;
    Delta d;
    TRY(make_delta(seq, par, false, s, d));
    if (s.rows > 0 && (!q || !k || !v || !gate || !beta || !y)) return CONV_ERR_NULL;
    const int e = esize(seq);
    const size_t need = delta_fwd_workspace(s, d, e == 2);
    TRY(check_workspace(workspace, workspace_bytes, need));
    const DeltaIn in{{q, ldq}, {k, ldk}, {v, ldv}, {gate, ldg}, {beta, ldb}};
    const Inputs i = inputs(in, d, s.rows, e);
    const int64_t ends = (int64_t)s.B * d.Hv * d.Dk * d.Dv, nb = (s.T + CONV_SCAN_BLOCK - 1) / CONV_SCAN_BLOCK;
    const Span sy{y, s.rows, s.C, ldy, e}, ss0 = dense(s0, ends, 4), ssT = dense(sT, ends, 4), ss = dense(states, ends * nb, 4),
        sws = dense(need ? workspace : nullptr, (int64_t)workspace_bytes, 1);
    TRY(check_align({i.q, i.k, i.v, i.g, i.b, sy, ss0, ssT, ss}));
    TRY(check_steps({i.q, i.k, i.v, i.g, i.b, sy}));
    TRY(check_alias({sy, ssT, ss, sws}, {i.q, i.k, i.v, i.g, i.b, ss0}));
    return to_status(launch_delta_fwd(s, d, e == 2, in, s0, RowsOut{y, ldy}, sT, states, workspace, (hipStream_t)stream));
}

size_t conv_delta_bwd_workspace_bytes(const conv_seq_t *seq, const conv_delta_t *par) {
    Seq s;
    Delta d;
    return make_delta(seq, par, false, s, d) == CONV_OK ? delta_bwd_workspace(s, d, esize(seq) == 2) : 0;
}

conv_status_t conv_delta_bwd(const conv_seq_t *seq, const conv_delta_t *par, const void *q, int64_t ldq, const void *k,
                             int64_t ldk, const void *v, int64_t ldv, const float *gate, int64_t ldg, const float *beta,
                             int64_t ldb, const float *states, const void *dy, int64_t lddy, const float *dsT, void *dq,
                             int64_t lddq, void *dk, int64_t lddk, void *dv, int64_t lddv, float *dgate, int64_t lddg,
                             float *dbeta, int64_t lddb, float *ds0, void *workspace, size_t workspace_bytes, void *stream) {
    Seq s;
    Delta d;
    TRY(make_delta(seq, par, false, s, d));
    if ((s.rows > 0 && (!q || !k || !v || !gate || !beta || !dy || !dq || !dk || !dv || !dgate || !dbeta)) ||
        (s.rows > 0 && s.T > 0 && !states))                 // no tokens, no states
        return CONV_ERR_NULL;
    const int e = esize(seq);
    const size_t need = delta_bwd_workspace(s, d, e == 2);
    TRY(check_workspace(workspace, workspace_bytes, need));
    const DeltaIn in{{q, ldq}, {k, ldk}, {v, ldv}, {gate, ldg}, {beta, ldb}};
    const Inputs i = inputs(in, d, s.rows, e);
    const int64_t ends = (int64_t)s.B * d.Hv * d.Dk * d.Dv, nb = (s.T + CONV_SCAN_BLOCK - 1) / CONV_SCAN_BLOCK;
    const int64_t wide = (int64_t)d.H * d.Dk;
    const Span sdy{dy, s.rows, s.C, lddy, e}, sdq{dq, s.rows, wide, lddq, e}, sdk{dk, s.rows, wide, lddk, e},
        sdv{dv, s.rows, s.C, lddv, e}, sdg{dgate, s.rows, d.Hv, lddg, 4}, sdb{dbeta, s.rows, d.Hv, lddb, 4},
        ss = dense(states, ends * nb, 4), sdT = dense(dsT, ends, 4), sd0 = dense(ds0, ends, 4),
        sws = dense(need ? workspace : nullptr, (int64_t)workspace_bytes, 1);
    TRY(check_align({i.q, i.k, i.v, i.g, i.b, ss, sdy, sdT, sdq, sdk, sdv, sdg, sdb, sd0}));
    TRY(check_steps({i.q, i.k, i.v, i.g, i.b, sdy, sdq, sdk, sdv, sdg, sdb}));
    TRY(check_alias({sdq, sdk, sdv, sdg, sdb, sd0, sws}, {i.q, i.k, i.v, i.g, i.b, ss, sdy, sdT}));
    return to_status(launch_delta_bwd(s, d, e == 2, in, states, Rows{dy, lddy}, dsT, RowsOut{dq, lddq}, RowsOut{dk, lddk},
                                      RowsOut{dv, lddv}, RowsOut{dgate, lddg}, RowsOut{dbeta, lddb}, ds0, workspace,
                                      (hipStream_t)stream));
}

conv_status_t conv_delta_step(const conv_seq_t *seq, const conv_delta_t *par, const void *q, int64_t ldq, const void *k,
                              int64_t ldk, const void *v, int64_t ldv, const float *gate, int64_t ldg, const float *beta,
                              int64_t ldb, float *S, void *y, int64_t ldy, void *stream) {
    Seq s;
    Delta d;
    TRY(make_delta(seq, par, true, s, d));
    if (!q || !k || !v || !gate || !beta || !S || !y) return CONV_ERR_NULL;
    const int e = esize(seq);
    const DeltaIn in{{q, ldq}, {k, ldk}, {v, ldv}, {gate, ldg}, {beta, ldb}};
    const Inputs i = inputs(in, d, s.B, e);
    const Span sS = dense(S, (int64_t)s.B * d.Hv * d.Dk * d.Dv, 4), sy{y, s.B, s.C, ldy, e};
    TRY(check_align({i.q, i.k, i.v, i.g, i.b, sS, sy}));
    TRY(check_steps({i.q, i.k, i.v, i.g, i.b, sy}));
    TRY(check_alias({sS, sy}, {i.q, i.k, i.v, i.g, i.b}));
    return to_status(launch_delta_step(s, d, e == 2, in, S, RowsOut{y, ldy}, (hipStream_t)stream));
}

}  // extern "C"
