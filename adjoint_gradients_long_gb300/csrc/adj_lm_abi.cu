// adj_lm_abi.cu -- the extern "C" entry points of the language-model operators: host-side
// validation and the launches.  The operations are documented in include/adj.h.
#include <math.h>

#include "adj_lin.cuh"
#include "adj_lm.cuh"

using namespace adj;

namespace {

#define ADJ_TRY(x)                                  \
    do {                                            \
        adj_status s_ = (x);                        \
        if (s_ != ADJ_OK) return s_;                \
    } while (0)

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// pointers that a call needs (null: refused) and pointers that it may go without
adj_status need(std::initializer_list<const void *> ps) {
    for (const void *p : ps) {
        if (!p) return ADJ_EINVAL;
        if (!aligned(p, 16)) return ADJ_EALIGN;
    }
    return ADJ_OK;
}
adj_status may(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (p && !aligned(p, 16)) return ADJ_EALIGN;
    return ADJ_OK;
}

adj_status check_lin(const adj_lin_dims *d, bool step) {
    if (!d) return ADJ_EINVAL;
    if (d->x_dtype != ADJ_F32 && d->x_dtype != ADJ_BF16) return ADJ_EDTYPE;
    if (d->B < 0 || (!step && d->T < 0) || d->H <= 0 || d->Hk <= 0 || d->H % d->Hk) return ADJ_ESHAPE;
    if (d->Dk < 8 || d->Dv < 8 || d->Dk > 128 || d->Dv > 128 || d->Dk % 8 || d->Dv % 8) return ADJ_ESHAPE;
    if (d->B > 65535 || d->H > 65535) return ADJ_ESHAPE;
    const int64_t vec = d->x_dtype == ADJ_BF16 ? 8 : 4, qk = int64_t(d->Hk) * d->Dk, vo = int64_t(d->H) * d->Dv;
    if (d->ldq < qk || d->ldk < qk || d->ldv < vo || d->ldo < vo) return ADJ_ESHAPE;
    if (d->ldq % vec || d->ldk % vec || d->ldv % vec || d->ldo % vec) return ADJ_EALIGN;
    // tensor maps: 32-bit token coordinates, 40-bit byte strides
    if (d->x_dtype == ADJ_BF16 && !step) {
        if (d->T >= (int64_t(1) << 31) || d->B * d->H * (d->T / 128 + 1) >= (int64_t(1) << 31)) return ADJ_ESHAPE;
        for (int64_t ld : {d->ldq, d->ldk, d->ldv, d->ldo})
            if (ld >= (int64_t(1) << 31) || d->T * ld >= (int64_t(1) << 39)) return ADJ_ESHAPE;
    }
    // grids: a block for 512 state values of every head, and one for every chunk
    if (d->B * d->H >= (int64_t(1) << 26) || (!step && d->T >= (int64_t(1) << 36))) return ADJ_ESHAPE;
    if (!isfinite(d->scale)) return ADJ_EINVAL;
    return ADJ_OK;
}

LinArgs lin_args(const adj_lin_dims *d) {
    LinArgs a{};
    a.B = d->B; a.T = d->T; a.H = d->H; a.Hk = d->Hk; a.Dk = d->Dk; a.Dv = d->Dv;
    a.NC = lin_chunks(d->T, d->x_dtype == ADJ_BF16);
    a.ldq = d->ldq; a.ldk = d->ldk; a.ldv = d->ldv; a.ldo = d->ldo;
    a.scale = d->scale;
    return a;
}

adj_status carve(const adj_lin_dims *d, bool bwd, LinArgs &a, void *ws, size_t ws_bytes) {
    if (!ws) return ADJ_EINVAL;
    if (!aligned(ws, 256)) return ADJ_EALIGN;
    const bool bf = d->x_dtype == ADJ_BF16;
    if (ws_bytes < WS_HEADER + lin_ws_bytes(a, bwd, bf)) return ADJ_EWORKSPACE;
    lin_ws_carve(a, bwd, bf, static_cast<char *>(ws) + WS_HEADER);
    return ADJ_OK;
}

inline adj_status done(cudaError_t e) { return e == cudaSuccess ? ADJ_OK : ADJ_ECUDA; }

}  // namespace

extern "C" {

size_t adj_lin_workspace_bytes(const adj_lin_dims *dims, int op) {
    if ((op != ADJ_OP_LIN_FWD && op != ADJ_OP_LIN_BWD) || check_lin(dims, false) != ADJ_OK) return 0;
    return WS_HEADER + lin_ws_bytes(lin_args(dims), op == ADJ_OP_LIN_BWD, dims->x_dtype == ADJ_BF16);
}

adj_status adj_lin_fwd(const adj_lin_dims *dims, const void *q, const void *k, const void *v, const float *g,
                       const float *s0, void *o, float *s1, void *ws, size_t ws_bytes, void *stream) {
    ADJ_TRY(check_lin(dims, false));
    if (dims->B * dims->T) ADJ_TRY(need({q, k, v, g, o}));
    ADJ_TRY(may({s0, s1}));
    LinArgs a = lin_args(dims);
    ADJ_TRY(carve(dims, false, a, ws, ws_bytes));
    if (a.B == 0) return ADJ_OK;
    a.q = q; a.k = k; a.v = v; a.g = g; a.s0 = s0; a.o = o; a.s1 = s1;
    return done(launch_lin_fwd(a, dims->x_dtype == ADJ_BF16, static_cast<unsigned *>(ws), static_cast<cudaStream_t>(stream)));
}

adj_status adj_lin_bwd(const adj_lin_dims *dims, const void *q, const void *k, const void *v, const float *g,
                       const float *s0, const void *go, const float *ds1, void *dq, void *dk, void *dv, float *dg,
                       float *ds0, void *ws, size_t ws_bytes, void *stream) {
    ADJ_TRY(check_lin(dims, false));
    if (dims->B * dims->T) ADJ_TRY(need({q, k, v, g, go, dq, dk, dv, dg}));
    ADJ_TRY(may({s0, ds1, ds0}));
    LinArgs a = lin_args(dims);
    ADJ_TRY(carve(dims, true, a, ws, ws_bytes));
    if (a.B == 0) return ADJ_OK;
    a.q = q; a.k = k; a.v = v; a.g = g; a.s0 = s0; a.go = go; a.ds1 = ds1;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.ds0 = ds0;
    return done(launch_lin_bwd(a, dims->x_dtype == ADJ_BF16, static_cast<unsigned *>(ws), static_cast<cudaStream_t>(stream)));
}

adj_status adj_lin_step(const adj_lin_dims *dims, const void *q, const void *k, const void *v, const float *g,
                        float *state, int64_t n_slots, const int32_t *slots, void *o, void *stream) {
    ADJ_TRY(check_lin(dims, true));
    if (dims->B) ADJ_TRY(need({q, k, v, g, state, o}));
    if (slots && !aligned(slots, 4)) return ADJ_EALIGN;
    if (n_slots < 0 || (!slots && n_slots < dims->B)) return ADJ_ESHAPE;
    if (dims->B == 0) return ADJ_OK;
    LinArgs a = lin_args(dims);
    a.q = q; a.k = k; a.v = v; a.g = g; a.o = o;
    return done(launch_lin_step(a, dims->x_dtype == ADJ_BF16, state, n_slots, slots, static_cast<cudaStream_t>(stream)));
}

adj_status adj_logprob(const adj_logprob_dims *d, const void *logits, const int64_t *targets, float *logp,
                       float *entropy, float *lse, int32_t *top_id, float *top_logp, const float *glp,
                       const float *gent, void *dlogits, void *stream) {
    if (!d) return ADJ_EINVAL;
    if (d->x_dtype != ADJ_F32 && d->x_dtype != ADJ_BF16) return ADJ_EDTYPE;
    if (d->N < 0 || d->N >= (int64_t(1) << 28) || d->V < 1 || d->V >= (int64_t(1) << 31) || d->ld < d->V) return ADJ_ESHAPE;
    if (d->top < 0 || d->top > ADJ_LOGPROB_MAX_TOP || d->top > d->V) return ADJ_ESHAPE;
    if (dlogits && d->ldd < d->V) return ADJ_ESHAPE;
    if (d->N == 0) return ADJ_OK;
    if (!logits) return ADJ_EINVAL;
    if ((logp || glp) && !targets) return ADJ_EINVAL;
    if ((d->top != 0) != (top_id != nullptr) || (d->top != 0) != (top_logp != nullptr)) return ADJ_EINVAL;
    if ((dlogits != nullptr) != (glp || gent)) return ADJ_EINVAL;
    if (dlogits == logits && d->ldd != d->ld) return ADJ_EINVAL;
    const uintptr_t el = d->x_dtype == ADJ_BF16 ? 2 : 4;
    if (!aligned(logits, el) || !aligned(dlogits, el) || !aligned(targets, 8)) return ADJ_EALIGN;
    for (const void *p : {(const void *)logp, (const void *)entropy, (const void *)lse, (const void *)top_id,
                          (const void *)top_logp, (const void *)glp, (const void *)gent})
        if (!aligned(p, 4)) return ADJ_EALIGN;
    LogprobArgs a{d->N, d->V, d->ld, d->ldd, d->top, logits, targets, logp, entropy, lse, top_id, top_logp, glp, gent, dlogits, 1, 0};
    return done(launch_logprob(a, d->x_dtype == ADJ_BF16, static_cast<cudaStream_t>(stream)));
}

size_t adj_clip_workspace_bytes(void) { return clip_ws_bytes(); }

adj_status adj_grad_clip(const adj_grad_seg *segs, int64_t nseg, float max_norm, float *out, void *ws,
                         size_t ws_bytes, void *stream) {
    if (nseg < 0) return ADJ_ESHAPE;
    if ((nseg && !segs) || !out || !ws) return ADJ_EINVAL;
    if (!(max_norm >= 0.f)) return ADJ_EINVAL;
    if (!aligned(out, 4) || !aligned(ws, 256)) return ADJ_EALIGN;
    if (ws_bytes < clip_ws_bytes()) return ADJ_EWORKSPACE;
    for (int64_t i = 0; i < nseg; ++i) {
        const adj_grad_seg &s = segs[i];
        if (s.n < 0 || s.n >= (int64_t(1) << 40)) return ADJ_ESHAPE;     // its chunks fit 31 bits
        if (s.dtype != ADJ_F32 && s.dtype != ADJ_BF16) return ADJ_EDTYPE;
        if (s.n && !s.src) return ADJ_EINVAL;
        const uintptr_t el = s.dtype == ADJ_BF16 ? 2 : 4;
        if (!aligned(s.src, el) || !aligned(s.dst, el)) return ADJ_EALIGN;
    }
    return done(launch_grad_clip(segs, nseg, max_norm, out, static_cast<char *>(ws), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
