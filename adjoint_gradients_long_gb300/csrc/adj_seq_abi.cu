// adj_seq_abi.cu -- the extern "C" entry points of the short convolution, the selective scan with states
// and sampling: host-side validation and the launches.  include/adj.h documents them.
#include <initializer_list>

#include "adj_seq.cuh"

using namespace adj;

namespace {

#define ADJ_TRY(x)                                  \
    do {                                            \
        adj_status s_ = (x);                        \
        if (s_ != ADJ_OK) return s_;                \
    } while (0)

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline adj_status done(cudaError_t e) { return e == cudaSuccess ? ADJ_OK : ADJ_ECUDA; }

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

// no output is an input
adj_status apart(std::initializer_list<const void *> outs, std::initializer_list<const void *> ins) {
    for (const void *o : outs)
        for (const void *i : ins)
            if (o && o == i) return ADJ_EINVAL;
    return ADJ_OK;
}

constexpr int64_t MOST_ROWS = int64_t(1) << 31;         // tokens of a call: their blocks fit a grid
constexpr int32_t MOST_CHANNELS = 1 << 20;

// sizes that both operators share; rows = B T of them where not packed
adj_status check_rows(int64_t B, int64_t T, int32_t P, int32_t packed, bool step, int64_t &rows) {
    rows = 0;
    if (B < 0 || B >= MOST_ROWS || (!step && (T < 0 || T >= MOST_ROWS))) return ADJ_ESHAPE;
    if (!step && packed != 0 && packed != 1) return ADJ_EINVAL;
    if (P < 8 || P % 8 || P > MOST_CHANNELS) return ADJ_ESHAPE;
    rows = step ? B : packed ? T : B * T;
    return rows < MOST_ROWS ? ADJ_OK : ADJ_ESHAPE;
}
adj_status check_pitch(int32_t dtype, std::initializer_list<std::pair<int64_t, int64_t>> lds) {
    const int64_t vec = dtype == ADJ_BF16 ? 8 : 4;
    for (const auto &l : lds)
        if (l.first < l.second || l.first >= (int64_t(1) << 31)) return ADJ_ESHAPE;
    for (const auto &l : lds)
        if (l.first % vec) return ADJ_EALIGN;
    return ADJ_OK;
}
adj_status check_offsets(int32_t packed, const int64_t *offsets) {
    if ((packed != 0) != (offsets != nullptr)) return ADJ_EINVAL;
    return aligned(offsets, 8) ? ADJ_OK : ADJ_EALIGN;
}
// a pool without entries needs no address: every slot is outside it
adj_status check_pool(int64_t B, const void *state, int64_t n_slots, const int32_t *slots) {
    ADJ_TRY(B && n_slots ? need({state}) : may({state}));
    if (slots && !aligned(slots, 4)) return ADJ_EALIGN;
    return n_slots < 0 || (!slots && n_slots < B) ? ADJ_ESHAPE : ADJ_OK;
}

adj_status check_conv(const adj_conv_dims *d, bool step, ConvArgs &a) {
    a = ConvArgs{};
    if (!d) return ADJ_EINVAL;
    if (d->x_dtype != ADJ_F32 && d->x_dtype != ADJ_BF16) return ADJ_EDTYPE;
    int64_t rows;
    ADJ_TRY(check_rows(d->B, d->T, d->P, d->packed, step, rows));
    if (d->W < 2 || d->W > 4) return ADJ_ESHAPE;
    if ((d->act != 0 && d->act != 1) || d->reserved) return ADJ_EINVAL;
    ADJ_TRY(check_pitch(d->x_dtype, {{d->ldx, d->P}, {d->ldy, d->P}}));
    a.q = Seqs{nullptr, d->B, step ? 1 : d->T, rows};
    a.ldx = d->ldx; a.ldy = d->ldy;
    a.P = d->P; a.W = d->W; a.act = d->act;
    // grids: a thread for every four channels of a step, blocks of 64 quads in their second dimension
    return !step || rows * (d->P / 4) < (int64_t(1) << 38) ? ADJ_OK : ADJ_ESHAPE;
}

adj_status check_ssm(const adj_ssm_dims *d, bool step, SsmArgs &a) {
    a = SsmArgs{};
    if (!d) return ADJ_EINVAL;
    if (d->x_dtype != ADJ_F32 && d->x_dtype != ADJ_BF16) return ADJ_EDTYPE;
    int64_t rows;
    ADJ_TRY(check_rows(d->B, d->T, d->P, d->packed, step, rows));
    if (d->N != 8 && d->N != 16 && d->N != 32 && d->N != 64) return ADJ_ESHAPE;
    ADJ_TRY(check_pitch(d->x_dtype, {{d->ldx, d->P}, {d->lddt, d->P}, {d->ldz, d->P}, {d->ldB, d->N}, {d->ldC, d->N}, {d->ldy, d->P}}));
    a.q = Seqs{nullptr, d->B, step ? 1 : d->T, rows};
    a.ldx = d->ldx; a.lddt = d->lddt; a.ldz = d->ldz; a.ldB = d->ldB; a.ldC = d->ldC; a.ldy = d->ldy;
    a.P = d->P; a.N = d->N;
    // grids: a thread for every four states of a step, for every four values of dB and dC
    return rows * int64_t(step ? d->P : 2) * (d->N / 4) < (int64_t(1) << 38) ? ADJ_OK : ADJ_ESHAPE;
}

adj_status plan(SsmArgs &a, bool bwd, void *ws, size_t ws_bytes) {
    if (!ws) return ADJ_EINVAL;
    if (!aligned(ws, 256)) return ADJ_EALIGN;
    return ws_bytes < WS_HEADER + ssm_plan(a, bwd, static_cast<char *>(ws) + WS_HEADER) ? ADJ_EWORKSPACE : ADJ_OK;
}

}  // namespace

extern "C" {

adj_status adj_conv_fwd(const adj_conv_dims *dims, const void *x, const float *w, const float *bias, const void *s0,
                        const int64_t *offsets, void *y, void *s1, void *stream) {
    ConvArgs a;
    ADJ_TRY(check_conv(dims, false, a));
    ADJ_TRY(check_offsets(dims->packed, offsets));
    if (a.q.rows) ADJ_TRY(need({x, w, y}));
    ADJ_TRY(may({bias, s0, s1}));
    ADJ_TRY(apart({y, s1}, {x, w, bias, s0, offsets}));
    a.q.off = offsets;
    a.x = x; a.w = w; a.bias = bias; a.s0 = s0; a.y = y; a.s1 = s1;
    if (a.q.B == 0) return ADJ_OK;
    return done(launch_conv_fwd(a, dims->x_dtype == ADJ_BF16, static_cast<cudaStream_t>(stream)));
}

size_t adj_conv_workspace_bytes(const adj_conv_dims *dims) {
    ConvArgs a;
    return check_conv(dims, false, a) == ADJ_OK ? WS_HEADER + conv_ws_bytes(a) : 0;
}

adj_status adj_conv_bwd(const adj_conv_dims *dims, const void *x, const float *w, const float *bias, const void *s0,
                        const int64_t *offsets, const void *go, const void *ds1, void *dx, float *dw, float *dbias,
                        void *ds0, void *ws, size_t ws_bytes, void *stream) {
    ConvArgs a;
    ADJ_TRY(check_conv(dims, false, a));
    ADJ_TRY(check_offsets(dims->packed, offsets));
    if (a.q.rows) ADJ_TRY(need({x, go, dx}));
    ADJ_TRY(need({w, dw}));
    ADJ_TRY(may({bias, s0, ds1, dbias, ds0}));
    ADJ_TRY(apart({dx, dw, dbias, ds0}, {x, w, bias, s0, offsets, go, ds1}));
    if (!ws) return ADJ_EINVAL;
    if (!aligned(ws, 256)) return ADJ_EALIGN;
    if (ws_bytes < WS_HEADER + conv_ws_bytes(a)) return ADJ_EWORKSPACE;
    a.q.off = offsets;
    a.x = x; a.w = w; a.bias = bias; a.s0 = s0; a.go = go; a.ds1 = ds1;
    a.dx = dx; a.dw = dw; a.dbias = dbias; a.ds0 = ds0;
    a.part = reinterpret_cast<float *>(static_cast<char *>(ws) + WS_HEADER);
    return done(launch_conv_bwd(a, dims->x_dtype == ADJ_BF16, static_cast<cudaStream_t>(stream)));
}

adj_status adj_conv_step(const adj_conv_dims *dims, const void *x, const float *w, const float *bias, void *state,
                         int64_t n_slots, const int32_t *slots, void *y, void *stream) {
    ConvArgs a;
    ADJ_TRY(check_conv(dims, true, a));
    if (a.q.B) ADJ_TRY(need({x, w, y}));
    ADJ_TRY(may({bias}));
    ADJ_TRY(check_pool(a.q.B, state, n_slots, slots));
    if (a.q.B == 0) return ADJ_OK;
    ADJ_TRY(apart({y, state}, {x, w, bias, slots}));
    if (y == state) return ADJ_EINVAL;
    a.x = x; a.w = w; a.bias = bias; a.y = y;
    return done(launch_conv_step(a, dims->x_dtype == ADJ_BF16, state, n_slots, slots, static_cast<cudaStream_t>(stream)));
}

size_t adj_ssm_workspace_bytes(const adj_ssm_dims *dims, int op) {
    SsmArgs a;
    if ((op != ADJ_OP_SSM_FWD && op != ADJ_OP_SSM_BWD) || check_ssm(dims, false, a) != ADJ_OK) return 0;
    return WS_HEADER + ssm_plan(a, op == ADJ_OP_SSM_BWD, nullptr);
}

adj_status adj_ssm_fwd(const adj_ssm_dims *dims, const void *x, const void *dt, const float *A, const void *Bm,
                       const void *Cm, const float *D, const void *z, const float *dt_bias, const float *s0,
                       const int64_t *offsets, void *y, float *s1, void *ws, size_t ws_bytes, void *stream) {
    SsmArgs a;
    ADJ_TRY(check_ssm(dims, false, a));
    ADJ_TRY(check_offsets(dims->packed, offsets));
    if (a.q.rows) ADJ_TRY(need({x, dt, A, Bm, Cm, y}));
    ADJ_TRY(may({D, z, dt_bias, s0, s1}));
    ADJ_TRY(apart({y, s1}, {x, dt, A, Bm, Cm, D, z, dt_bias, s0, offsets}));
    ADJ_TRY(plan(a, false, ws, ws_bytes));
    if (a.q.B == 0) return ADJ_OK;
    a.q.off = offsets;
    a.x = x; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.D = D; a.z = z; a.bias = dt_bias; a.s0 = s0; a.y = y; a.s1 = s1;
    return done(launch_ssm_fwd(a, dims->x_dtype == ADJ_BF16, static_cast<cudaStream_t>(stream)));
}

adj_status adj_ssm_bwd(const adj_ssm_dims *dims, const void *x, const void *dt, const float *A, const void *Bm,
                       const void *Cm, const float *D, const void *z, const float *dt_bias, const float *s0,
                       const int64_t *offsets, const void *go, const float *ds1, void *dx, void *ddt, float *dA,
                       void *dB, void *dC, float *dD, void *dz, float *ddt_bias, float *ds0, void *ws,
                       size_t ws_bytes, void *stream) {
    SsmArgs a;
    ADJ_TRY(check_ssm(dims, false, a));
    ADJ_TRY(check_offsets(dims->packed, offsets));
    if (a.q.rows) ADJ_TRY(need({x, dt, Bm, Cm, go, dx, ddt, dB, dC}));
    ADJ_TRY(need({A, dA}));
    if ((z != nullptr) != (dz != nullptr)) return ADJ_EINVAL;
    ADJ_TRY(may({D, z, dt_bias, s0, ds1, dD, dz, ddt_bias, ds0}));
    ADJ_TRY(apart({dx, ddt, dA, dB, dC, dD, dz, ddt_bias, ds0}, {x, dt, A, Bm, Cm, D, z, dt_bias, s0, offsets, go, ds1}));
    ADJ_TRY(plan(a, true, ws, ws_bytes));
    a.q.off = offsets;
    a.x = x; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.D = D; a.z = z; a.bias = dt_bias; a.s0 = s0;
    a.go = go; a.ds1 = ds1; a.dx = dx; a.ddt = ddt; a.dA = dA; a.dB = dB; a.dC = dC; a.dD = dD; a.dz = dz;
    a.dbias = ddt_bias; a.ds0 = ds0;
    return done(launch_ssm_bwd(a, dims->x_dtype == ADJ_BF16, static_cast<cudaStream_t>(stream)));
}

adj_status adj_ssm_step(const adj_ssm_dims *dims, const void *x, const void *dt, const float *A, const void *Bm,
                        const void *Cm, const float *D, const void *z, const float *dt_bias, float *state,
                        int64_t n_slots, const int32_t *slots, void *y, void *stream) {
    SsmArgs a;
    ADJ_TRY(check_ssm(dims, true, a));
    if (a.q.B) ADJ_TRY(need({x, dt, A, Bm, Cm, y}));
    ADJ_TRY(may({D, z, dt_bias}));
    ADJ_TRY(check_pool(a.q.B, state, n_slots, slots));
    if (a.q.B == 0) return ADJ_OK;
    ADJ_TRY(apart({y, state}, {x, dt, A, Bm, Cm, D, z, dt_bias, slots}));
    if (y == state) return ADJ_EINVAL;
    a.x = x; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.D = D; a.z = z; a.bias = dt_bias; a.y = y;
    return done(launch_ssm_step(a, dims->x_dtype == ADJ_BF16, state, n_slots, slots, static_cast<cudaStream_t>(stream)));
}

adj_status adj_sample(const adj_sample_dims *d, const void *logits, const float *u, const float *temperature,
                      const int32_t *top_k, const float *top_p, const float *min_p, int64_t *token, float *logp,
                      void *stream) {
    if (!d) return ADJ_EINVAL;
    if (d->x_dtype != ADJ_F32 && d->x_dtype != ADJ_BF16) return ADJ_EDTYPE;
    if (d->N < 0 || d->N >= (int64_t(1) << 28) || d->V < 1 || d->V > ADJ_SAMPLE_MAX_V || d->ld < d->V) return ADJ_ESHAPE;
    if (d->reserved) return ADJ_EINVAL;
    if (d->N == 0) return ADJ_OK;
    if (!logits || !u || !token) return ADJ_EINVAL;
    if (!aligned(logits, d->x_dtype == ADJ_BF16 ? 2 : 4) || !aligned(token, 8)) return ADJ_EALIGN;
    for (const void *p : {(const void *)u, (const void *)temperature, (const void *)top_k, (const void *)top_p,
                          (const void *)min_p, (const void *)logp})
        if (!aligned(p, 4)) return ADJ_EALIGN;
    const SampleArgs a{d->N, d->V, d->ld, logits, u, temperature, top_p, min_p, top_k, token, logp};
    return done(launch_sample(a, d->x_dtype == ADJ_BF16, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
