// seq_api.cpp -- the extern "C" entry points of the operators over sequences of
// tokens, of the layer norm and of the optimiser step.  As in conv_api.cpp, every argument is
// checked on the host before any HIP call.
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <vector>

#include "conv_fwd.h"
#include "norm_internal.h"
#include "optim_internal.h"
#include "seq_checks.h"
#include "seq_internal.h"

using namespace convfwd;

namespace {

// The recurrence has 512 threads to a workgroup and a launch fewer than 2^32: the last of the sizes above is
// one too many, and so is the one before it where a workgroup more fills rows.
conv_status_t make_scan(const conv_seq_t *q, Seq &s) {
    const conv_status_t st = make_seq(q, false, s);
    if (st != CONV_OK) return st;
    return (s.rows / CONV_SCAN_BLOCK + s.B) * ((s.C + 63) / 64) + s.fill >= kMaxBlocks ? CONV_ERR_OVERFLOW : CONV_OK;
}

bool bad_causal(int K, int silu) { return K < 1 || K > 8 || (silu != 0 && silu != 1); }

}  // namespace

extern "C" {

// ---- causal convolution ----

conv_status_t conv_causal_fwd(const conv_seq_t *seq, int K, int silu, const void *x, int64_t ldx, const void *w,
                              const float *bias, const void *state, void *y, int64_t ldy, void *state_out, void *stream) {
    Seq s;
    TRY(make_seq(seq, false, s));
    if (!w || (s.rows > 0 && (!x || !y))) return CONV_ERR_NULL;
    if (bad_causal(K, silu)) return CONV_ERR_PARAM;
    const int e = esize(seq);
    const int64_t carried = (int64_t)s.B * (K - 1) * s.C;
    const Span sx{x, s.rows, s.C, ldx, e}, sy{y, s.rows, s.C, ldy, e}, sw = dense(w, (int64_t)s.C * K, e),
        sb = dense(bias, s.C, 4), s0 = dense(state, carried, e), s1 = dense(state_out, carried, e);
    TRY(check_align({sx, sy, sw, sb, s0, s1}));
    TRY(check_alias({sy, s1}, {sx, sw, sb, s0}));
    return to_status(convfwd::launch_causal_fwd(s, e == 2, K, silu, x, ldx, w, bias, state, y, ldy, state_out,
                                                (hipStream_t)stream));
}

size_t conv_causal_bwd_workspace_bytes(const conv_seq_t *seq, int K) {
    Seq s;
    if (make_seq(seq, false, s) != CONV_OK || bad_causal(K, 0)) return 0;
    return (size_t)convfwd::causal_bwd_workspace_floats(s, K) * 4;
}

conv_status_t conv_causal_bwd(const conv_seq_t *seq, int K, int silu, const void *x, int64_t ldx, const void *w,
                              const float *bias, const void *state, const void *dy, int64_t lddy, void *dx,
                              int64_t lddx, float *dw, float *db, void *dstate, void *workspace, size_t workspace_bytes,
                              void *stream) {
    Seq s;
    TRY(make_seq(seq, false, s));
    if (!w || !dw || (s.rows > 0 && (!x || !dy || !dx))) return CONV_ERR_NULL;
    if (bad_causal(K, silu)) return CONV_ERR_PARAM;
    TRY(check_workspace(workspace, workspace_bytes, (size_t)convfwd::causal_bwd_workspace_floats(s, K) * 4));
    const int e = esize(seq);
    const int64_t carried = (int64_t)s.B * (K - 1) * s.C;
    const Span sx{x, s.rows, s.C, ldx, e}, sdy{dy, s.rows, s.C, lddy, e}, sdx{dx, s.rows, s.C, lddx, e},
        sw = dense(w, (int64_t)s.C * K, e), sb = dense(bias, s.C, 4), s0 = dense(state, carried, e),
        sdw = dense(dw, (int64_t)s.C * K, 4), sdb = dense(db, s.C, 4), sds = dense(dstate, carried, e),
        sws = dense(workspace, (int64_t)workspace_bytes, 1);
    TRY(check_align({sx, sdy, sdx, sw, sb, s0, sdw, sdb, sds}));
    TRY(check_alias({sdx, sdw, sdb, sds, sws}, {sx, sdy, sw, sb, s0}));
    return to_status(convfwd::launch_causal_bwd(s, e == 2, K, silu, x, ldx, w, bias, state, dy, lddy, dx, lddx, dw, db,
                                                dstate, (float *)workspace, (hipStream_t)stream));
}

conv_status_t conv_causal_step(const conv_seq_t *seq, int K, int silu, const void *x, int64_t ldx, const void *w,
                               const float *bias, void *state, void *y, int64_t ldy, void *stream) {
    Seq s;
    TRY(make_seq(seq, true, s));
    if (!x || !w || !y || (K > 1 && !state)) return CONV_ERR_NULL;
    if (bad_causal(K, silu)) return CONV_ERR_PARAM;
    const int e = esize(seq);
    const Span sx{x, s.B, s.C, ldx, e}, sy{y, s.B, s.C, ldy, e}, sw = dense(w, (int64_t)s.C * K, e),
        sb = dense(bias, s.C, 4), s0 = dense(state, (int64_t)s.B * (K - 1) * s.C, e);
    TRY(check_align({sx, sy, sw, sb, s0}));
    TRY(check_alias({sy, s0}, {sx, sw, sb}));
    return to_status(convfwd::launch_causal_step(s, e == 2, K, silu, x, ldx, w, bias, state, y, ldy, (hipStream_t)stream));
}

// ---- gated recurrence ----

size_t conv_scan_fwd_workspace_bytes(const conv_seq_t *seq) {
    Seq s;
    return make_scan(seq, s) == CONV_OK ? convfwd::scan_fwd_workspace(s) : 0;
}

conv_status_t conv_scan_fwd(const conv_seq_t *seq, float scale, const void *x, int64_t ldx, const void *gate, int64_t ldg,
                            const void *inp, int64_t ldi, const float *decay, const float *h0, void *y, int64_t ldy,
                            float *hT, float *states, void *workspace, size_t workspace_bytes, void *stream) {
    Seq s;
    TRY(make_scan(seq, s));
    if (!decay || (s.rows > 0 && (!x || !gate || !inp || !y))) return CONV_ERR_NULL;
    if (!(scale >= 0.f) || isinf(scale)) return CONV_ERR_PARAM;
    const size_t need = convfwd::scan_fwd_workspace(s);
    TRY(check_workspace(workspace, workspace_bytes, need));
    const int e = esize(seq);
    const int64_t ends = (int64_t)s.B * s.C, nb = (s.T + CONV_SCAN_BLOCK - 1) / CONV_SCAN_BLOCK;
    const Span sx{x, s.rows, s.C, ldx, e}, sg{gate, s.rows, s.C, ldg, e}, si{inp, s.rows, s.C, ldi, e},
        sy{y, s.rows, s.C, ldy, e}, sd = dense(decay, s.C, 4), s0 = dense(h0, ends, 4), sT = dense(hT, ends, 4),
        ss = dense(states, ends * nb, 4), sws = dense(need ? workspace : nullptr, (int64_t)workspace_bytes, 1);
    TRY(check_align({sx, sg, si, sy, sd, s0, sT, ss}));
    TRY(check_alias({sy, sT, ss, sws}, {sx, sg, si, sd, s0}));
    return to_status(convfwd::launch_scan_fwd(s, e == 2, scale, x, ldx, gate, ldg, inp, ldi, decay, h0, y, ldy, hT, states,
                                              workspace, (hipStream_t)stream));
}

size_t conv_scan_bwd_workspace_bytes(const conv_seq_t *seq) {
    Seq s;
    return make_scan(seq, s) == CONV_OK ? convfwd::scan_bwd_workspace(s) : 0;
}

conv_status_t conv_scan_bwd(const conv_seq_t *seq, float scale, const void *x, int64_t ldx, const void *gate, int64_t ldg,
                            const void *inp, int64_t ldi, const float *decay, const float *states, const void *dy,
                            int64_t lddy, const float *dhT, void *dx, int64_t lddx, void *dgate, int64_t lddg, void *dinp,
                            int64_t lddi, float *ddecay, float *dh0, void *workspace, size_t workspace_bytes, void *stream) {
    Seq s;
    TRY(make_scan(seq, s));
    if (!decay || !ddecay || (s.rows > 0 && (!x || !gate || !inp || !dy || !dx || !dgate || !dinp)) ||
        (s.rows > 0 && s.T > 0 && !states))                 // no tokens, no states
        return CONV_ERR_NULL;
    if (!(scale >= 0.f) || isinf(scale)) return CONV_ERR_PARAM;
    TRY(check_workspace(workspace, workspace_bytes, convfwd::scan_bwd_workspace(s)));
    const int e = esize(seq);
    const int64_t ends = (int64_t)s.B * s.C, nb = (s.T + CONV_SCAN_BLOCK - 1) / CONV_SCAN_BLOCK;
    const Span sx{x, s.rows, s.C, ldx, e}, sg{gate, s.rows, s.C, ldg, e}, si{inp, s.rows, s.C, ldi, e},
        sdy{dy, s.rows, s.C, lddy, e}, sd = dense(decay, s.C, 4), ss = dense(states, ends * nb, 4), sT = dense(dhT, ends, 4),
        sdx{dx, s.rows, s.C, lddx, e}, sdg{dgate, s.rows, s.C, lddg, e}, sdi{dinp, s.rows, s.C, lddi, e},
        sdd = dense(ddecay, s.C, 4), sd0 = dense(dh0, ends, 4), sws = dense(workspace, (int64_t)workspace_bytes, 1);
    TRY(check_align({sx, sg, si, sdy, sd, ss, sT, sdx, sdg, sdi, sdd, sd0}));
    TRY(check_alias({sdx, sdg, sdi, sdd, sd0, sws}, {sx, sg, si, sdy, sd, ss, sT}));
    return to_status(convfwd::launch_scan_bwd(s, e == 2, scale, x, ldx, gate, ldg, inp, ldi, decay, states, dy, lddy, dhT, dx,
                                              lddx, dgate, lddg, dinp, lddi, ddecay, dh0, workspace, (hipStream_t)stream));
}

conv_status_t conv_scan_step(const conv_seq_t *seq, float scale, const void *x, int64_t ldx, const void *gate, int64_t ldg,
                             const void *inp, int64_t ldi, const float *decay, float *h, void *y, int64_t ldy, void *stream) {
    Seq s;
    TRY(make_seq(seq, true, s));
    if (!x || !gate || !inp || !decay || !h || !y) return CONV_ERR_NULL;
    if (!(scale >= 0.f) || isinf(scale)) return CONV_ERR_PARAM;
    const int e = esize(seq);
    const Span sx{x, s.B, s.C, ldx, e}, sg{gate, s.B, s.C, ldg, e}, si{inp, s.B, s.C, ldi, e}, sy{y, s.B, s.C, ldy, e},
        sd = dense(decay, s.C, 4), sh = dense(h, (int64_t)s.B * s.C, 4);
    TRY(check_align({sx, sg, si, sy, sd, sh}));
    TRY(check_alias({sy, sh}, {sx, sg, si, sd}));
    return to_status(convfwd::launch_scan_step(s, e == 2, scale, x, ldx, gate, ldg, inp, ldi, decay, h, y, ldy,
                                               (hipStream_t)stream));
}

// ---- layer norm ----

static conv_status_t check_norm(int dtype, int64_t rows, int C) {
    if ((dtype != CONV_OUT_F32 && dtype != CONV_OUT_BF16) || rows < 0 || C < 1) return CONV_ERR_PARAM;
    return rows >= kMaxRows || C > kMaxChannels ? CONV_ERR_OVERFLOW : CONV_OK;
}

conv_status_t conv_norm_fwd(int dtype, int64_t rows, int C, float eps, const void *x, int64_t ldx, const float *weight,
                            const float *bias, void *y, int64_t ldy, float *mean, float *rstd, void *stream) {
    TRY(check_norm(dtype, rows, C));
    if (rows > 0 && (!x || !y)) return CONV_ERR_NULL;
    if (!(eps >= 0.f) || isinf(eps)) return CONV_ERR_PARAM;
    const int e = dtype == CONV_OUT_BF16 ? 2 : 4;
    const Span sx{x, rows, C, ldx, e}, sy{y, rows, C, ldy, e}, sw = dense(weight, C, 4), sb = dense(bias, C, 4),
        sm = dense(mean, rows, 4), sr = dense(rstd, rows, 4);
    TRY(check_align({sx, sy, sw, sb, sm, sr}));
    TRY(check_alias({sy, sm, sr}, {sx, sw, sb}));
    return to_status(convfwd::launch_norm_fwd(rows, C, e == 2, eps, x, ldx, weight, bias, y, ldy, mean, rstd, (hipStream_t)stream));
}

size_t conv_norm_bwd_workspace_bytes(int dtype, int64_t rows, int C) {
    if (check_norm(dtype, rows, C) != CONV_OK) return 0;
    return (size_t)convfwd::norm_bwd_workspace_floats(rows, C, dtype == CONV_OUT_BF16) * 4;
}

conv_status_t conv_norm_bwd(int dtype, int64_t rows, int C, const void *x, int64_t ldx, const float *weight, const float *mean,
                            const float *rstd, const void *dy, int64_t lddy, void *dx, int64_t lddx, float *dweight,
                            float *dbias, void *workspace, size_t workspace_bytes, void *stream) {
    TRY(check_norm(dtype, rows, C));
    if (rows > 0 && (!x || !mean || !rstd || !dy || !dx)) return CONV_ERR_NULL;
    const int e = dtype == CONV_OUT_BF16 ? 2 : 4;
    const size_t need = dweight || dbias ? (size_t)convfwd::norm_bwd_workspace_floats(rows, C, e == 2) * 4 : 0;
    TRY(check_workspace(workspace, workspace_bytes, need));
    const Span sx{x, rows, C, ldx, e}, sdy{dy, rows, C, lddy, e}, sdx{dx, rows, C, lddx, e}, sw = dense(weight, C, 4),
        sm = dense(mean, rows, 4), sr = dense(rstd, rows, 4), sdw = dense(dweight, C, 4), sdb = dense(dbias, C, 4),
        sws = dense(need ? workspace : nullptr, (int64_t)workspace_bytes, 1);
    TRY(check_align({sx, sdy, sdx, sw, sm, sr, sdw, sdb}));
    TRY(check_alias({sdx, sdw, sdb, sws}, {sx, sdy, sw, sm, sr}));
    return to_status(convfwd::launch_norm_bwd(rows, C, e == 2, x, ldx, weight, mean, rstd, dy, lddy, dx, lddx, dweight, dbias,
                                              (float *)workspace, (hipStream_t)stream));
}

// ---- optimiser ----

conv_status_t conv_adamw_step(const conv_adamw_t *o, const conv_adamw_tensor_t *tensors, int count, void *stream) {
    if (!o || (count > 0 && !tensors)) return CONV_ERR_NULL;
    const auto finite = [](double v) { return v >= 0 && v <= 3.4e38; };      // and not NaN
    if (count < 0 || o->step < 1 || !(o->beta1 >= 0 && o->beta1 < 1) || !(o->beta2 >= 0 && o->beta2 < 1) ||
        !finite(o->lr) || !finite(o->eps) || (o->bits != 8 && o->bits != 32) ||
        (o->grad_dtype != CONV_OUT_F32 && o->grad_dtype != CONV_OUT_BF16) || (uintptr_t)o->grad_scale % 4)
        return CONV_ERR_PARAM;
    const int ge = o->grad_dtype == CONV_OUT_BF16 ? 2 : 4, me = o->bits == 8 ? 1 : 4;
    std::vector<AdamwTensor> list;
    try {
        list.reserve(count);
    } catch (...) {
        return CONV_ERR_OVERFLOW;
    }
    for (int i = 0; i < count; ++i) {
        const conv_adamw_tensor_t &t = tensors[i];
        if (t.n < 0 || !finite(t.weight_decay)) return CONV_ERR_PARAM;
        if (t.n >= INT64_C(2147483648)) return CONV_ERR_OVERFLOW;
        if (t.n == 0) continue;
        if (!t.p || !t.g || !t.m || !t.v || (me == 1 && (!t.m_scale || !t.v_scale))) return CONV_ERR_NULL;
        const int64_t nq = me == 1 ? (t.n + 255) / 256 : 0;
        const Span p = dense(t.p, t.n, 4), g = dense(t.g, t.n, ge), m = dense(t.m, t.n, me), v = dense(t.v, t.n, me),
                   ms = dense(t.m_scale, nq, 4), vs = dense(t.v_scale, nq, 4), c = dense(t.copy, t.n, 2);
        TRY(check_align({p, g, m, v, ms, vs, c}));
        TRY(check_alias({p, m, v, ms, vs, c}, {g, dense(o->grad_scale, 1, 4)}));
        AdamwTensor a;
        a.p = t.p, a.g = t.g, a.m = t.m, a.v = t.v, a.m_scale = t.m_scale, a.v_scale = t.v_scale, a.copy = t.copy;
        a.n = t.n;
        a.keep = (float)(1.0 - o->lr * (double)t.weight_decay);
        a.key = o->seed * 0x632be5abu + (uint32_t)o->step * 0x2545f491u + (uint32_t)i * 0x7feb352du;
        a.first = a.pad = 0;
        list.push_back(a);
    }
    AdamwHyper h;
    h.b1 = (float)o->beta1, h.ob1 = (float)(1.0 - o->beta1);
    h.b2 = (float)o->beta2, h.ob2 = (float)(1.0 - o->beta2);
    h.lr_c1 = (float)(o->lr / (1.0 - pow(o->beta1, (double)o->step)));
    h.inv_sqrt_c2 = (float)(1.0 / sqrt(1.0 - pow(o->beta2, (double)o->step)));
    // An eps below the normal numbers counts as the smallest of these: the hardware's reciprocal would make 0 * inf
    // of 0 / eps.  A v above 0 has a root of 2^-75 or more, which does not notice either.
    h.eps = o->eps > 0 && o->eps < FLT_MIN ? FLT_MIN : (float)o->eps;
    h.pad = 0.f;
    h.grad_scale = o->grad_scale;
    return to_status(convfwd::launch_adamw(h, list.data(), (int)list.size(), me == 1 ? convfwd::kAdamw8 : convfwd::kAdamw32,
                                           ge == 2, (hipStream_t)stream));
}

conv_status_t conv_adamw_state_values(const conv_adamw_tensor_t *tensors, int count, float *const *m_out,
                                      float *const *v_out, void *stream) {
    if (count > 0 && (!tensors || !m_out || !v_out)) return CONV_ERR_NULL;
    if (count < 0) return CONV_ERR_PARAM;
    std::vector<AdamwTensor> list;
    try {
        list.reserve(count);
    } catch (...) {
        return CONV_ERR_OVERFLOW;
    }
    for (int i = 0; i < count; ++i) {
        const conv_adamw_tensor_t &t = tensors[i];
        if (t.n < 0) return CONV_ERR_PARAM;
        if (t.n >= INT64_C(2147483648)) return CONV_ERR_OVERFLOW;
        if (t.n == 0) continue;
        if (!t.m || !t.v || !t.m_scale || !t.v_scale || !m_out[i] || !v_out[i]) return CONV_ERR_NULL;
        const int64_t nq = (t.n + 255) / 256;
        const Span m = dense(t.m, t.n, 1), v = dense(t.v, t.n, 1), ms = dense(t.m_scale, nq, 4), vs = dense(t.v_scale, nq, 4),
                   mo = dense(m_out[i], t.n, 4), vo = dense(v_out[i], t.n, 4);
        TRY(check_align({ms, vs, mo, vo}));
        TRY(check_alias({mo, vo}, {m, v, ms, vs}));
        AdamwTensor a = {};
        a.p = m_out[i], a.copy = (uint16_t *)v_out[i], a.m = t.m, a.v = t.v, a.m_scale = t.m_scale, a.v_scale = t.v_scale;
        a.n = t.n;
        list.push_back(a);
    }
    return to_status(convfwd::launch_adamw(AdamwHyper{}, list.data(), (int)list.size(), convfwd::kAdamwValues, false,
                                           (hipStream_t)stream));
}

}  // extern "C"
