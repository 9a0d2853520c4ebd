// adj_seq.cuh -- what the short convolution and the selective scan share: sequences in a run of
// tokens, vectors of eight channels, packed pairs of fp32, and the launchers.
#pragma once
#include <type_traits>

#include "adj_internal.cuh"

namespace adj {

inline int64_t seq_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The sequences of a call (include/adj.h, "Sequences").  Offsets are held to [0, rows], and an index
// that a search returns to [0, B), whatever the array holds.
struct Seqs {
    const int64_t *off;         // null: B sequences of T tokens each
    int64_t B, T, rows;

    __device__ __forceinline__ int64_t at(int64_t i) const {
        const int64_t v = off[i];
        return v < 0 ? 0 : v > rows ? rows : v;
    }
    __device__ __forceinline__ int64_t begin(int64_t b) const { return off ? at(b) : b * T; }
    __device__ __forceinline__ int64_t end(int64_t b) const { return off ? at(b + 1) : (b + 1) * T; }
    // the sequence that holds token t, or -1
    __device__ __forceinline__ int64_t find(int64_t t) const {
        if (!off) return t < rows ? int64_t(uint32_t(t) / uint32_t(T)) : -1;       // rows < 2^31
        int64_t lo = 0, hi = B + 1;                     // entries below lo are at most t, those from hi on larger
        while (lo < hi) {
            const int64_t mid = (lo + hi) >> 1;
            if (at(mid) <= t) lo = mid + 1;
            else hi = mid;
        }
        return lo <= B ? lo - 1 : -1;
    }
};

// ---------------------------------------------------------------- eight channels
template <class T>
struct Raw8;
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = __ldg(reinterpret_cast<const float4 *>(p));
        b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};
template <>
struct Raw8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};

// ---------------------------------------------------------------- four channels, as they are stored
template <class T>
struct Raw4;
template <>
struct Raw4<float> {
    float4 v;
    __device__ __forceinline__ void load(const float *p) { v = __ldg(reinterpret_cast<const float4 *>(p)); }
    __device__ __forceinline__ void load_own(const float *p) { v = *reinterpret_cast<const float4 *>(p); }   // not by way of the read-only cache
    __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<float4 *>(p) = v; }
    __device__ __forceinline__ void zero() { v = f4(0.f); }
    __device__ __forceinline__ float4 get() const { return v; }
};
template <>
struct Raw4<__nv_bfloat16> {
    uint2 v;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = __ldg(reinterpret_cast<const uint2 *>(p)); }
    __device__ __forceinline__ void load_own(const __nv_bfloat16 *p) { v = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint2 *>(p) = v; }
    __device__ __forceinline__ void zero() { v = make_uint2(0, 0); }
    __device__ __forceinline__ float4 get() const {
        return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                           __uint_as_float(v.y & 0xFFFF0000u));
    }
};

// ---------------------------------------------------------------- functions of one value
__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float SEQ_LOG2E = 1.4426950408889634f, SEQ_LN2 = 0.6931471805599453f;
// 1 / (1 + e^-x): the exponential overflows to infinity below -88, whose reciprocal is zero
__device__ __forceinline__ float sigmoid_f(float x) { return fast_rcp(1.f + fast_exp2(-x * SEQ_LOG2E)); }

__device__ __forceinline__ float4 sigmoid4(float4 v) {
    return make_float4(sigmoid_f(v.x), sigmoid_f(v.y), sigmoid_f(v.z), sigmoid_f(v.w));
}

// ---------------------------------------------------------------- pairs of fp32 in one instruction
typedef unsigned long long pair_t;
__device__ __forceinline__ pair_t pk(float x, float y) {
    pair_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void upk(pair_t v, float &x, float &y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ pair_t mul2(pair_t a, pair_t b) {
    pair_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ pair_t fma2(pair_t a, pair_t b, pair_t c) {
    pair_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ pair_t add2(pair_t a, pair_t b) {
    pair_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ pair_t exp2_2(pair_t v) {
    float x, y;
    upk(v, x, y);
    return pk(fast_exp2(x), fast_exp2(y));
}

// log(1 + e^v) = max(v, 0) + log1p(e), e = e^-|v|.  What the exponent's product loses is made up for, so that
// small steps keep 23 bits; log1p(e) / e is a polynomial of degree 9 on 0 to 1, fitted by least squares
// reweighted towards its largest error, 5e-9.  Below -100 it is zero; a NaN stays one.
__device__ __forceinline__ pair_t softplus_2(float x, float y) {
    const float lx = fmaxf(-fabsf(x), -100.f), ly = fmaxf(-fabsf(y), -100.f);
    float mx, my;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(mx) : "f"(x));
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(my) : "f"(y));
    const pair_t u = pk(lx, ly), p = mul2(u, pk(SEQ_LOG2E, SEQ_LOG2E));
    pair_t e = exp2_2(p);
    constexpr float H = -0.693147182464599609375f, L = 1.904654323148236017e-9f;
    e = fma2(e, fma2(p, pk(L, L), fma2(p, pk(H, H), u)), e);
    constexpr float C[10] = {1.f, -0.4999990165233612f, 0.3332996368408203f, -0.24954132735729218f, 0.19675934314727783f,
                             -0.153055801987648f, 0.10603633522987366f, -0.05695932358503342f, 0.019851351156830788f,
                             -0.003244000254198909f};
    pair_t c = pk(C[9], C[9]);
#pragma unroll
    for (int i = 8; i >= 0; --i) c = fma2(c, e, pk(C[i], C[i]));
    return fma2(e, c, pk(mx, my));
}
__device__ __forceinline__ float softplus_f(float v) {
    float x, y;
    upk(softplus_2(v, v), x, y);
    return x;
}

// ---------------------------------------------------------------- calls, resolved on the host
struct ConvArgs {
    Seqs q;
    int64_t ldx, ldy;
    int P, W, act;
    const void *x, *s0, *go, *ds1;
    const float *w, *bias;
    void *y, *s1, *dx, *ds0;
    float *dw, *dbias;
    float *part;                // backward: [blocks of tokens][W+1][P]
};
size_t conv_ws_bytes(const ConvArgs &a);
cudaError_t launch_conv_fwd(const ConvArgs &a, bool bf16, cudaStream_t st);
cudaError_t launch_conv_bwd(const ConvArgs &a, bool bf16, cudaStream_t st);
cudaError_t launch_conv_step(const ConvArgs &a, bool bf16, void *state, int64_t n_slots, const int32_t *slots,
                             cudaStream_t st);

struct SsmArgs {
    Seqs q;
    int64_t ldx, lddt, ldz, ldB, ldC, ldy;
    int P, N;
    const void *x, *dt, *Bm, *Cm, *z, *go;
    const float *A, *D, *bias, *s0, *ds1;
    void *y, *dx, *ddt, *dB, *dC, *dz;
    float *s1, *dA, *dD, *dbias, *ds0;
    // workspace
    int64_t nseg, seglen;       // the tokens are cut into nseg segments of seglen (the last may be shorter)
    float *seg;                 // [nseg][P][N]: the state a segment makes from nothing, then the one that enters it
    float *step;                // [nseg][P]: sum of its steps; -1: a sequence begins in it
    float *adj;                 // [nseg][P][N]: the same of the adjoint state, from the right
    float *tile, *tstep;        // [tiles][P][N], [tiles][P]: state and steps from the segment's start to each tile
    float *bc;                  // [blocks of channels][rows][2 N]: partial sums of dB and dC
    float *par;                 // [nseg][P][N+2]: partial sums of dA, then of dD and ddt_bias
};
// cuts the tokens, and lays out the workspace from `base` (null: sizes alone); its bytes
size_t ssm_plan(SsmArgs &a, bool bwd, void *base);
cudaError_t launch_ssm_fwd(const SsmArgs &a, bool bf16, cudaStream_t st);
cudaError_t launch_ssm_bwd(const SsmArgs &a, bool bf16, cudaStream_t st);
cudaError_t launch_ssm_step(const SsmArgs &a, bool bf16, float *state, int64_t n_slots, const int32_t *slots,
                            cudaStream_t st);

struct SampleArgs {
    int64_t N, V, ld;
    const void *logits;
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int64_t *token;
    float *logp;
};
cudaError_t launch_sample(const SampleArgs &a, bool bf16, cudaStream_t st);

}  // namespace adj
