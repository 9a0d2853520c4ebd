// adj_lm.cu -- log probabilities of given tokens (with entropy, top alternatives and the
// gradient) and clipping gradients by their global norm.  include/adj.h defines them.
#include <algorithm>

#include "adj_lm.cuh"
#include "adj_profile.cuh"

namespace adj {
namespace {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16 bytes of T as floats
template <class T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(uint4 u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    static __device__ __forceinline__ float get(float x) { return x; }
    static __device__ __forceinline__ float put(float x) { return x; }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<uint32_t *>(&v);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};

// An array of n values of any alignment as 16-byte vectors: vector i holds the elements
// i * N - shift .. + N, of which the first and the last vector may lie partly outside.
template <class T>
struct Ragged {
    static constexpr int N = Vec<T>::N;
    T *p;
    int64_t n;
    int shift;
    __device__ Ragged(T *p_, int64_t n_) : p(p_), n(n_), shift(int((reinterpret_cast<uintptr_t>(p_) & 15u) / sizeof(T))) {}
    __device__ int64_t vectors() const { return (n + shift + N - 1) / N; }
    __device__ bool whole(int64_t i) const { return i * N >= shift && (i + 1) * N - shift <= n; }
    __device__ uint4 raw(int64_t i) const { return __ldg(reinterpret_cast<const uint4 *>(p + (i * N - shift))); }
    __device__ void load(int64_t i, float (&x)[N], float fill) const {
        if (whole(i)) {
            Vec<T>::unpack(raw(i), x);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int64_t j = i * N - shift + e;
                x[e] = j >= 0 && j < n ? Vec<T>::get(p[j]) : fill;
            }
        }
    }
    // aligned: p has the alignment that the vectors were cut for
    __device__ void store(int64_t i, int cut, const float (&x)[N]) const {
        const int64_t j0 = i * N - cut;
        if (shift == cut && j0 >= 0 && j0 + N <= n) {
            *reinterpret_cast<uint4 *>(p + j0) = Vec<T>::pack(x);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (j0 + e >= 0 && j0 + e < n) p[j0 + e] = Vec<T>::put(x[e]);
        }
    }
};

// ---------------------------------------------------------------- log probabilities
constexpr int LPT = 512;        // threads of a row
constexpr int CAND = 1024;      // candidates for the top list

// Order of the top list as unsigned integers: NaN above +inf, the zeros equal.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
// (key, index) as one number: larger is better, among equal keys the lower index
__device__ __forceinline__ uint64_t rank_key(uint32_t key, uint32_t idx) { return (uint64_t(key) << 32) | uint32_t(~idx); }

// Running softmax statistics in powers of two: m the largest x seen, s = sum 2^(d), t = sum
// 2^(d) d with d = (x - m) log2 e.
struct Stat {
    float m, s, t;
};
// Distances from m in powers of two.  One multiply-add each, on the rounded m log2 e, which
// every use of the same m shares; beyond 2^127 that product would overflow and the difference is
// taken first.  A row with nothing but masked values is measured from zero.
struct Ref {
    float m, m2;
    bool far;
    __device__ __forceinline__ explicit Ref(float m_) : m(m_ == -INFINITY ? 0.f : m_), m2(m * LOG2E), far(fabsf(m) > 1.7e38f) {}
    __device__ __forceinline__ float operator()(float x) const { return far ? (x - m) * LOG2E : fmaf(x, LOG2E, -m2); }
    __device__ __forceinline__ float from(const Ref &o) const { return far || o.far ? (o.m - m) * LOG2E : o.m2 - m2; }
    // log(sum) of a sum s = 2^l2s measured from m, and a value's logarithm less that
    __device__ __forceinline__ float natural(float l2s) const { return far ? m + l2s * LN2 : (m2 + l2s) * LN2; }
    __device__ __forceinline__ float logp(float x, float l2s) const {
        return far ? (x - m) - l2s * LN2 : (fmaf(x, LOG2E, -m2) - l2s) * LN2;
    }
};
__device__ __forceinline__ Stat join(Stat a, Stat b) {
    const float m = fmaxf(a.m, b.m);
    const Ref r(m);
    Stat o{m, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const Stat &x = k ? b : a;
        if (x.s == 0.f) continue;                        // nothing, or only masked values
        const float d = r.from(Ref(x.m)), e = ex2(d);
        o.s = fmaf(x.s, e, o.s);
        if (e != 0.f) o.t += e * fmaf(x.s, d, x.t);
    }
    return o;
}

template <class T, bool GRAD>
__global__ __launch_bounds__(LPT) void k_logprob(const LogprobArgs a) {
    constexpr int N = Vec<T>::N;
    __shared__ Stat red[LPT / 32];
    __shared__ Stat all;
    __shared__ uint64_t cand[CAND];
    __shared__ int n_cand;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const Ragged<T> x(const_cast<T *>(static_cast<const T *>(a.logits)) + row * a.ld, a.V);
    const int64_t nv = x.vectors();

    Stat st{-INFINITY, 0.f, 0.f};
    for (int64_t i = tid; i < nv; i += LPT) {
        float v[N];
        x.load(i, v, -INFINITY);
        float m = v[0];
#pragma unroll
        for (int e = 1; e < N; ++e) m = fmaxf(m, v[e]);
        if (m > st.m) {
            if (st.s != 0.f) {
                const float d = Ref(m).from(Ref(st.m)), f = ex2(d);
                st.t = f == 0.f ? 0.f : f * fmaf(st.s, d, st.t);
                st.s *= f;
            }
            st.m = m;
        }
        const Ref r(st.m);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float d = r(v[e]), p = ex2(d);
            st.s += p;
            if (p != 0.f) st.t = fmaf(p, d, st.t);       // a masked value has d = -inf
        }
    }
    const float own_max = st.m;
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        Stat o;
        o.m = __shfl_xor_sync(~0u, st.m, d);
        o.s = __shfl_xor_sync(~0u, st.s, d);
        o.t = __shfl_xor_sync(~0u, st.t, d);
        st = join(st, o);
    }
    if ((tid & 31) == 0) red[tid >> 5] = st;
    if (tid == 0) n_cand = 0;
    __syncthreads();
    if (tid == 0) {
        Stat s = red[0];
        for (int w = 1; w < LPT / 32; ++w) s = join(s, red[w]);
        all = s;
    }
    __syncthreads();
    const Ref ref(all.m);
    const float s = all.s, l2s = log2f(s);
    const bool empty = s == 0.f;
    const float lse = empty ? -INFINITY : ref.natural(l2s), ent = empty ? 0.f : (l2s - all.t / s) * LN2;
    const int64_t y = a.targets ? a.targets[row] : -1;
    const bool scored = y >= 0 && y < a.V;
    if (tid == 0) {
        if (a.lse) a.lse[row] = lse;
        if (a.entropy) a.entropy[row] = ent;
        if (a.logp)
            a.logp[row] = !scored ? 0.f : empty ? -INFINITY : ref.logp(Vec<T>::get(x.p[y]), l2s);
    }
    if (a.top) {
        // Lower bound of the top-th largest: the top-th largest of the threads' own maxima, to 16
        // bits of its key.  Only threads at or above it read their values again.
        const bool slow_row = s != s;                    // NaN or +inf: own_max says too little
        const uint32_t key = order_key(own_max);
        uint32_t bound = 0;
        for (int b = 31; b >= 16; --b) {
            const uint32_t c = bound | (1u << b);
            if (__syncthreads_count(key >= c) >= a.top) bound = c;
        }
        if (!slow_row && key >= bound)
            for (int64_t i = tid; i < nv; i += LPT)
                for (int e = 0; e < N; ++e) {
                    const int64_t j = i * N - x.shift + e;
                    if (j < 0 || j >= a.V) continue;
                    const uint32_t k = order_key(Vec<T>::get(x.p[j]));
                    if (k < bound) continue;
                    const int at = atomicAdd(&n_cand, 1);
                    if (at < CAND) cand[at] = rank_key(k, uint32_t(j));
                }
        __syncthreads();
        const int n = n_cand;
        int32_t *id = a.top_id + row * a.top;
        float *lp = a.top_logp + row * a.top;
        auto put = [&](int r, uint64_t c) {
            const uint32_t j = ~uint32_t(c);
            id[r] = int32_t(j);
            lp[r] = empty ? -INFINITY : ref.logp(Vec<T>::get(x.p[j]), l2s);
        };
        if (!slow_row && n <= CAND) {
            for (int i = tid; i < n; i += LPT) {
                int r = 0;
                for (int k = 0; k < n; ++k) r += cand[k] > cand[i];
                if (r < a.top) put(r, cand[i]);
            }
        } else {
            // many equal values, or NaN: the best of those after the last one taken, `top` times
            uint64_t last = ~uint64_t(0);
            for (int r = 0; r < a.top; ++r) {
                uint64_t best = 0;
                for (int64_t j = tid; j < a.V; j += LPT) {
                    const uint64_t c = rank_key(order_key(Vec<T>::get(x.p[j])), uint32_t(j));
                    if (c < last && c > best) best = c;
                }
#pragma unroll
                for (int d = 16; d; d >>= 1) best = max(best, __shfl_xor_sync(~0u, best, d));
                if ((tid & 31) == 0) cand[tid >> 5] = best;
                __syncthreads();
                for (int w = 0; w < LPT / 32; ++w) best = max(best, cand[w]);
                __syncthreads();
                if (tid == 0) put(r, best);
                last = best;
            }
        }
    }
    if (GRAD) {
        const float gl = scored && !empty && a.glp ? a.glp[row] : 0.f, ge = a.gent ? a.gent[row] : 0.f;
        const float inv = empty ? 0.f : 1.f / s;
        const Ragged<T> out(static_cast<T *>(a.dlogits) + row * a.ldd, a.V);
        if (a.top) __syncthreads();                      // in place: the top list has been read
        for (int64_t i = tid; i < nv; i += LPT) {
            float v[N];
            x.load(i, v, -INFINITY);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float d = ref(v[e]), p = ex2(d) * inv;
                float g = -gl * p;
                if (p != 0.f) g -= ge * p * fmaf(d - l2s, LN2, ent);
                if (i * N - x.shift + e == y && scored) g += gl;
                v[e] = g;
            }
            out.store(i, x.shift, v);
        }
    }
}

// ---------------------------------------------------------------- clipping
constexpr int CT = 256;         // threads of a block
constexpr int CLIP_CHUNK = 16384;   // bytes of a chunk

template <int MAXS>
struct ClipSegs {
    int n, first_group;         // first_group: the total starts with this group of tensors
    float max_norm;
    int64_t chunks;
    const void *src[MAXS];
    void *dst[MAXS];
    int64_t len[MAXS];
    int first[MAXS];            // a tensor's first chunk
    uint8_t bf16[MAXS];
};

template <int MAXS>
__device__ __forceinline__ int seg_of(const ClipSegs<MAXS> &g, int64_t c) {
    int lo = 0, hi = g.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (g.first[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <class T>
__device__ __forceinline__ float chunk_square(const void *src, int64_t n, int64_t c) {
    constexpr int N = Vec<T>::N, PER = CLIP_CHUNK / 16 / CT;
    const Ragged<T> x(const_cast<T *>(static_cast<const T *>(src)), n);
    const int64_t nv = x.vectors(), i0 = c * (CLIP_CHUNK / 16) + threadIdx.x;
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        const int64_t i = i0 + u * CT;
        if (i >= nv) break;
        float v[N];
        x.load(i, v, 0.f);
#pragma unroll
        for (int e = 0; e < N; ++e) s[e & 1] = fmaf(v[e], v[e], s[e & 1]);
    }
    return s[0] + s[1];
}

template <class T>
__device__ __forceinline__ void chunk_scale(const void *src, void *dst, int64_t n, int64_t c, float f) {
    constexpr int N = Vec<T>::N, PER = CLIP_CHUNK / 16 / CT;
    const Ragged<T> x(const_cast<T *>(static_cast<const T *>(src)), n), y(static_cast<T *>(dst), n);
    const int64_t nv = x.vectors(), i0 = c * (CLIP_CHUNK / 16) + threadIdx.x;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        const int64_t i = i0 + u * CT;
        if (i >= nv) break;
        float v[N];
        x.load(i, v, 0.f);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] *= f;
        y.store(i, x.shift, v);
    }
}

// Sum of squares: a block takes the chunks blockIdx.x, + gridDim.x, ...; the last block to
// finish adds the blocks' sums in their order.
template <int MAXS>
__global__ __launch_bounds__(CT) void k_clip_norm(const __grid_constant__ ClipSegs<MAXS> g, double *part, double *total,
                                                  unsigned *ticket, float *out) {
    __shared__ double red[CT / 32];
    __shared__ bool last;
    double sum = 0.0;
    for (int64_t c = blockIdx.x; c < g.chunks; c += gridDim.x) {
        const int s = seg_of(g, c);
        const int64_t k = c - g.first[s];
        sum += g.bf16[s] ? chunk_square<__nv_bfloat16>(g.src[s], g.len[s], k) : chunk_square<float>(g.src[s], g.len[s], k);
    }
    auto block_sum = [&](double v) {
#pragma unroll
        for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        double r = 0.0;
        for (int w = 0; w < CT / 32; ++w) r += red[w];
        __syncthreads();
        return r;
    };
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        part[blockIdx.x] = sum;
        __threadfence();
        last = atomicInc(ticket, gridDim.x - 1) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    double v = 0.0;
    for (int b = threadIdx.x; b < int(gridDim.x); b += CT) v += __ldcg(part + b);
    v = block_sum(v);
    if (threadIdx.x == 0) {
        if (!g.first_group) v += *total;
        *total = v;
        const float norm = float(sqrt(v)), c = g.max_norm / (norm + ADJ_CLIP_EPS);
        out[0] = norm;
        out[1] = c > 1.f ? 1.f : c;                      // NaN stays NaN
    }
}

template <int MAXS>
__global__ __launch_bounds__(CT) void k_clip_scale(const __grid_constant__ ClipSegs<MAXS> g, const float *out) {
    const float f = out[1];
    for (int64_t c = blockIdx.x; c < g.chunks; c += gridDim.x) {
        const int s = seg_of(g, c);
        if (!g.dst[s] || (g.dst[s] == g.src[s] && f == 1.f)) continue;
        const int64_t k = c - g.first[s];
        if (g.bf16[s]) chunk_scale<__nv_bfloat16>(g.src[s], g.dst[s], g.len[s], k, f);
        else chunk_scale<float>(g.src[s], g.dst[s], g.len[s], k, f);
    }
}

constexpr int CLIP_GRID = 152 * 8;

template <int MAXS>
int64_t fill(ClipSegs<MAXS> &t, const adj_grad_seg *segs, int64_t i, int64_t nseg) {
    t.n = 0;
    t.chunks = 0;
    for (; i < nseg && t.n < MAXS; ++i) {
        if (segs[i].n == 0) continue;
        const bool bf = segs[i].dtype == ADJ_BF16;
        const int64_t bytes = (reinterpret_cast<uintptr_t>(segs[i].src) & 15u) + segs[i].n * (bf ? 2 : 4);
        if (t.chunks + cdiv(bytes, CLIP_CHUNK) >= (int64_t(1) << 31)) break;
        t.src[t.n] = segs[i].src;
        t.dst[t.n] = segs[i].dst;
        t.len[t.n] = segs[i].n;
        t.first[t.n] = int(t.chunks);
        t.bf16[t.n] = bf;
        t.chunks += cdiv(bytes, CLIP_CHUNK);
        ++t.n;
    }
    return i;
}

template <int MAXS>
cudaError_t clip(const adj_grad_seg *segs, int64_t nseg, float max_norm, float *out, char *ws, cudaStream_t st) {
    double *part = reinterpret_cast<double *>(ws + WS_HEADER), *total = part + CLIP_GRID;
    unsigned *ticket = reinterpret_cast<unsigned *>(ws) + 2;
    ClipSegs<MAXS> t;
    t.max_norm = max_norm;
    for (int pass = 0; pass < 2; ++pass) {
        int64_t i = 0;
        t.first_group = 1;
        do {
            i = fill(t, segs, i, nseg);
            const unsigned grid = unsigned(std::max<int64_t>(1, std::min<int64_t>(t.chunks, CLIP_GRID)));
            ProfScope ps(pass ? K_CLIP_SCALE : K_CLIP_NORM, st);
            if (pass == 0) k_clip_norm<MAXS><<<grid, CT, 0, st>>>(t, part, total, ticket, out);
            else k_clip_scale<MAXS><<<grid, CT, 0, st>>>(t, out);
            const cudaError_t e = cudaGetLastError();
            if (e != cudaSuccess) return e;
            t.first_group = 0;
        } while (i < nseg);
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_logprob(const LogprobArgs &a, bool bf16, cudaStream_t st) {
    ProfScope ps(K_LOGPROB, st);
    const unsigned grid = unsigned(a.N);
    if (bf16) {
        if (a.dlogits) k_logprob<__nv_bfloat16, true><<<grid, LPT, 0, st>>>(a);
        else k_logprob<__nv_bfloat16, false><<<grid, LPT, 0, st>>>(a);
    } else {
        if (a.dlogits) k_logprob<float, true><<<grid, LPT, 0, st>>>(a);
        else k_logprob<float, false><<<grid, LPT, 0, st>>>(a);
    }
    return cudaGetLastError();
}

size_t clip_ws_bytes() { return WS_HEADER + (CLIP_GRID + 1) * sizeof(double); }

cudaError_t launch_grad_clip(const adj_grad_seg *segs, int64_t nseg, float max_norm, float *out, char *ws,
                             cudaStream_t st) {
    return nseg <= 64 ? clip<64>(segs, nseg, max_norm, out, ws, st) : clip<1000>(segs, nseg, max_norm, out, ws, st);
}

}  // namespace adj
