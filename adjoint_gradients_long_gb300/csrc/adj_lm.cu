// adj_lm.cu -- log probabilities of given tokens (with entropy, top alternatives and the
// gradient) and clipping gradients by their global norm.  include/adj.h defines them.
#include <algorithm>
#include <atomic>

#include "adj_lm.cuh"
#include "adj_profile.cuh"

namespace adj {
namespace {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// 16 bytes of T as floats
template <class T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static constexpr uint32_t LOW = 0xFF800000u;         // minus infinity, N of them
    static __device__ __forceinline__ float largest(uint4 u) {
        return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
    }
    // values below -2^18 as -2^18 (NaN stays)
    static __device__ __forceinline__ uint32_t floor1(uint32_t w) {
        float y;
        asm("max.NaN.f32 %0, %1, 0fC8800000;" : "=f"(y) : "f"(__uint_as_float(w)));
        return __float_as_uint(y);
    }
    static __device__ __forceinline__ uint4 floored(uint4 u) {
        return make_uint4(floor1(u.x), floor1(u.y), floor1(u.z), floor1(u.w));
    }
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
    static constexpr uint32_t LOW = 0xFF80FF80u;
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    static __device__ __forceinline__ float largest(uint4 u) {
        const uint32_t m = max2(max2(u.x, u.y), max2(u.z, u.w));
        return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t floor2(uint32_t w) {
        uint32_t d;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(w), "r"(0xC880C880u));
        return d;
    }
    static __device__ __forceinline__ uint4 floored(uint4 u) {
        return make_uint4(floor2(u.x), floor2(u.y), floor2(u.z), floor2(u.w));
    }
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
// One pass over the row with the running maximum, sum and entropy sum of its softmax; the
// gradient's second pass finds the row in L2.  Bound by the row's bytes, then by the instructions
// of a value (12 for both passes in bf16).  A row is cut over a cluster of 1 to 8 blocks: when the
// rows in flight would not stay in L2 otherwise, and when there are too few rows to fill the SMs.
// The blocks' statistics and top lists are joined through distributed shared memory, in rank order.
//
// Measured, loss with gradient of 8192 x 32768 bf16 (1.07 GB): 179 us, 0.89 of the
// copy bandwidth; with the row kept in shared memory, three blocks of 512 an SM, 227 us (the
// occupancy is worth more than the L2 reads).  Scoring 2048 x 50001 fp32: 86 us, 0.70; the
// same in bf16 57 us, 0.53; loss with gradient in fp32 (2.15 GB) 362 us, 0.87.
constexpr int LPT = 256;        // threads of a block
constexpr int LPB = 6;          // blocks an SM
constexpr int CAND = 512;       // candidates for the top list
constexpr int LPU = 4;          // vectors in flight a thread
// bytes of a row that one block takes when the gradient reads them again: 152 x 6 such parts are
// 64 MB, half of L2
constexpr int64_t ROW_PART = 72 * 1024;

// Order of the top list as unsigned integers: NaN above +inf, the zeros equal.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return k == 0xFFFFFFFFu ? NAN : __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}
// (key, index) as one number: larger is better, among equal keys the lower index
__device__ __forceinline__ uint64_t rank_key(uint32_t key, uint32_t idx) { return (uint64_t(key) << 32) | uint32_t(~idx); }

// Running softmax statistics in powers of two: m the largest x seen, s = sum 2^(d), t = sum
// 2^(d) d with d = (x - m) log2 e.
struct Stat {
    float m, s, t;
};
// Distances from m in powers of two.  One multiply-add each, on m2 = m log2 e as rounded, which
// every use of the same m shares: the distance of m itself is m2's rounding error, off().  It grows with
// m (and 2^off overflows from 1e10 on), so past FAR_FROM, where it may reach 0.003, the difference is
// taken before the product.  A row with nothing but masked values is measured from zero.
constexpr float FAR_FROM = 65536.f;
struct Ref {
    float m, m2;
    bool far;
    __device__ __forceinline__ explicit Ref(float m_) : m(m_ == -INFINITY ? 0.f : m_), m2(m * LOG2E), far(fabsf(m) > FAR_FROM) {}
    template <bool FAR>
    __device__ __forceinline__ float at(float x) const { return FAR ? (x - m) * LOG2E : fmaf(x, LOG2E, -m2); }
    // what a distance from here exceeds (x - m) log2 e by
    __device__ __forceinline__ float off() const { return far ? 0.f : fmaf(m, LOG2E, -m2); }
    // from here to another reference, at most at this one
    __device__ __forceinline__ float from(const Ref &o) const {
        return far || o.far ? fmaf(o.m - m, LOG2E, off() - o.off()) : o.m2 - m2;
    }
    // log(sum) of a sum s = 2^l2s measured from m, and a value's logarithm less that: the difference
    // first, which no value of fp32 overflows but where the result does
    __device__ __forceinline__ float natural(float l2s) const { return m + (l2s - off()) * LN2; }
    __device__ __forceinline__ float logp(float x, float l2s) const { return (x - m) - (l2s - off()) * LN2; }
};
__device__ __forceinline__ Stat join(Stat a, Stat b) {
    const float m = fmaxf(a.m, b.m);
    const Ref r(m);
    Stat o{m, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const Stat &x = k ? b : a;
        if (x.s == 0.f) continue;                        // nothing, or only masked values
        const float d = r.from(Ref(x.m)), e = fast_exp2(d);
        o.s = fmaf(x.s, e, o.s);
        if (e != 0.f) o.t += e * fmaf(x.s, d, x.t);
    }
    return o;
}

__device__ __forceinline__ uint32_t rank_in_cluster() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void meet(int blocks) {
    if (blocks == 1) __syncthreads();
    else asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// another block's copy of an object in shared memory
template <class X>
__device__ __forceinline__ X peer(const X *own, uint32_t rank) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(own)), b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(a), "r"(rank));
    union {
        X x;
        uint32_t w[sizeof(X) / 4];
    } u;
#pragma unroll
    for (int i = 0; i < int(sizeof(X) / 4); ++i)
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(u.w[i]) : "r"(b + 4 * i) : "memory");
    return u.x;
}

// The statistics of a whole warp, in every lane: the largest maximum, then plain sums.
__device__ __forceinline__ Stat warp_join(Stat x) {
    float m = x.m;
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
    if (x.s != 0.f) {
        const float d = Ref(m).from(Ref(x.m)), f = fast_exp2(d);
        x.t = f == 0.f ? 0.f : f * fmaf(x.s, d, x.t);
        x.s *= f;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        x.s += __shfl_xor_sync(~0u, x.s, d);
        x.t += __shfl_xor_sync(~0u, x.t, d);
    }
    x.m = m;
    return x;
}

// 2^distance times the distance is zero for a masked value, but minus infinity times zero would
// be NaN.  Values are raised to -2^18 first (half an instruction each in bf16), whose power of two is
// zero from every reference that is not far: distances stay above -5e5, so that the gradient's
// c0 + c1 distance is finite for cotangents up to 7e32 times the row's sum.  From a far one (FAR) the
// distance is held to -200, below which its power of two is zero.
template <class T, bool FAR>
__device__ __forceinline__ void distances(uint4 raw, const Ref &r, float (&d)[Vec<T>::N], float (&p)[Vec<T>::N]) {
    Vec<T>::unpack(FAR ? raw : Vec<T>::floored(raw), d);
#pragma unroll
    for (int e = 0; e < Vec<T>::N; ++e) {
        d[e] = r.at<FAR>(d[e]);
        p[e] = fast_exp2(d[e]);
        if (FAR) d[e] = fmaxf(d[e], -200.f);
    }
}

template <class T, bool FAR, int U>
__device__ __forceinline__ void add_up(Stat &st, const uint4 (&raw)[U]) {
    constexpr int N = Vec<T>::N;
    const Ref r(st.m);
    float s[2] = {0.f, 0.f}, t[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float d[N], p[N];
        distances<T, FAR>(raw[u], r, d, p);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            s[e & 1] += p[e];
            t[e & 1] = fmaf(p[e], d[e], t[e & 1]);
        }
    }
    st.s += s[0] + s[1];
    st.t += t[0] + t[1];
}

template <class T, int U>
__device__ __forceinline__ void take(Stat &st, const uint4 (&raw)[U]) {
    float m = Vec<T>::largest(raw[0]);
#pragma unroll
    for (int u = 1; u < U; ++u) m = fmaxf(m, Vec<T>::largest(raw[u]));
    if (m > st.m) {
        if (st.s != 0.f) {
            const float d = Ref(m).from(Ref(st.m)), f = fast_exp2(d);
            st.t = f == 0.f ? 0.f : f * fmaf(st.s, d, st.t);
            st.s *= f;
        }
        st.m = m;
    }
    if (Ref(st.m).far) add_up<T, true>(st, raw);
    else add_up<T, false>(st, raw);
}

// g = p (c0 + c1 d) of one vector, p = 2^d
template <class T, bool FAR>
__device__ __forceinline__ uint4 slope(uint4 raw, const Ref &ref, float c0, float c1) {
    float d[Vec<T>::N], p[Vec<T>::N];
    distances<T, FAR>(raw, ref, d, p);
#pragma unroll
    for (int e = 0; e < Vec<T>::N; ++e) d[e] = p[e] * fmaf(c1, d[e], c0);
    return Vec<T>::pack(d);
}

template <class T, bool GRAD>
__global__ __launch_bounds__(LPT, LPB) void k_logprob(const LogprobArgs a) {
    constexpr int N = Vec<T>::N;
    __shared__ Stat red[LPT / 32], mine;
    __shared__ uint64_t cand[CAND], best_of[ADJ_LOGPROB_MAX_TOP];
    __shared__ uint32_t keys[LPT], bound_;
    __shared__ int n_cand;
    const int tid = threadIdx.x, blocks = a.blocks;
    const uint32_t rank = blocks > 1 ? rank_in_cluster() : 0u;
    const int64_t row = blockIdx.x >> a.log_blocks;
    const Ragged<T> x(const_cast<T *>(static_cast<const T *>(a.logits)) + row * a.ld, a.V);
    // this block's vectors v0 .. v0 + nv of the row; the first and the last of a row may lie partly
    // outside it and are fetched value by value
    const int all_v = int(x.vectors()), per = (all_v + blocks - 1) >> a.log_blocks, v0 = int(rank) * per, nv = max(0, min(all_v - v0, per));
    const bool odd_first = nv > 0 && !x.whole(v0), odd_last = nv > 1 && !x.whole(v0 + nv - 1);
    const int w0 = odd_first ? 1 : 0, w1 = nv - (odd_last ? 1 : 0);
    const uint4 *src = reinterpret_cast<const uint4 *>(x.p - x.shift) + v0;
    const int64_t y = a.targets ? a.targets[row] : -1;
    const bool scored = y >= 0 && y < a.V;
    // before any block of the row may write its gradient over it
    const float at_y = scored ? Vec<T>::get(x.p[y]) : 0.f;
    auto fetch = [&](int i) {                            // any vector of this block
        if (i >= w0 && i < w1) return __ldg(src + i);
        float v[N];
        x.load(v0 + i, v, -INFINITY);
        return Vec<T>::pack(v);
    };

    Stat st{-INFINITY, 0.f, 0.f};
    int i = w0 + tid;
    for (; i + (LPU - 1) * LPT < w1; i += LPU * LPT) {
        uint4 raw[LPU];
#pragma unroll
        for (int u = 0; u < LPU; ++u) raw[u] = __ldg(src + i + u * LPT);
        take<T, LPU>(st, raw);
    }
    // the rest, then the vectors at the row's ends (threads 0 and 1)
    const int end = tid == 0 && odd_first ? 0 : tid == 1 && odd_last ? nv - 1 : nv;
    for (i = i < w1 ? i : end; i < nv; i = i + LPT < w1 && i != end ? i + LPT : i == end ? nv : end) {
        const uint4 raw[1] = {fetch(i)};
        take<T, 1>(st, raw);
    }
    const float own_max = st.m;
    st = warp_join(st);
    if ((tid & 31) == 0) red[tid >> 5] = st;
    if (tid == 0) n_cand = 0;
    __syncthreads();
    if (tid < 32) {
        st = warp_join(tid < LPT / 32 ? red[tid] : Stat{-INFINITY, 0.f, 0.f});
        if (tid == 0) mine = st;
    }
    if (a.top) {
        // This block's part of the top list.  A lower bound of its top-th largest value: the top-th
        // largest of the threads' own maxima, to 12 bits of its key (an eighth of a power of two).  Only
        // threads at or above it read their values again.
        const uint32_t key = order_key(own_max);
        keys[tid] = key;
        __syncthreads();
        const bool odd = mine.s != mine.s;               // NaN or +inf: own_max says too little
        if (tid < 32) {
            uint32_t k[LPT / 32], bound = 0;
#pragma unroll
            for (int w = 0; w < LPT / 32; ++w) k[w] = keys[w * 32 + tid];
#pragma unroll 1
            for (int b = 31; b >= 20; --b) {
                const uint32_t c = bound | (1u << b);
                int n = 0;
#pragma unroll
                for (int w = 0; w < LPT / 32; ++w) n += k[w] >= c;
                if (__reduce_add_sync(~0u, n) >= a.top) bound = c;
            }
            if (tid == 0) bound_ = bound;
        }
        __syncthreads();
        const uint32_t bound = bound_;
        auto offer = [&](int i) {
            float v[N];
            Vec<T>::unpack(fetch(i), v);
            const int64_t j0 = int64_t(v0 + i) * N - x.shift;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int64_t j = j0 + e;
                const uint32_t k = order_key(v[e]);
                if (k < bound || j < 0 || j >= a.V) continue;
                const int at = atomicAdd(&n_cand, 1);
                if (at < CAND) cand[at] = rank_key(k, uint32_t(j));
            }
        };
        if (!odd) {
            // a thread's values are read again by its whole warp: few threads qualify
#pragma unroll 1
            for (uint32_t m = __ballot_sync(~0u, key >= bound); m; m &= m - 1) {
                const int t = (tid & ~31) + __ffs(m) - 1;
#pragma unroll 1
                for (int i = w0 + t + (tid & 31) * LPT; i < w1; i += 32 * LPT) offer(i);
                if (t == tid && tid == 0 && odd_first) offer(0);
                if (t == tid && tid == 1 && odd_last) offer(nv - 1);
            }
        }
        if (tid < a.top) best_of[tid] = 0;               // fewer values than places
        __syncthreads();
        const int n = n_cand;
        if (!odd && n <= CAND) {
            // the order of the candidates is the threads'; their ranks are not
            for (int i = tid; i < n; i += LPT) {
                int r = 0;
#pragma unroll 1
                for (int k = 0; k < n; ++k) r += cand[k] > cand[i];
                if (r < a.top) best_of[r] = cand[i];
            }
        } else {
            // many equal values, or NaN: the best of those after the last one taken, `top` times
            uint64_t last = ~uint64_t(0);
            for (int r = 0; r < a.top; ++r) {
                uint64_t best = 0;
                for (int i = tid; i < nv; i += LPT) {
                    float v[N];
                    Vec<T>::unpack(fetch(i), v);
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const int64_t j = int64_t(v0 + i) * N - x.shift + e;
                        const uint64_t c = rank_key(order_key(v[e]), uint32_t(j));
                        if (j >= 0 && j < a.V && c < last && c > best) best = c;
                    }
                }
#pragma unroll
                for (int d = 16; d; d >>= 1) best = max(best, __shfl_xor_sync(~0u, best, d));
                __syncthreads();
                if ((tid & 31) == 0) cand[tid >> 5] = best;
                __syncthreads();
                for (int w = 0; w < LPT / 32; ++w) best = max(best, cand[w]);
                if (tid == 0) best_of[r] = best;
                last = best;
            }
        }
    }
    meet(blocks);
    Stat all = mine;
    if (blocks > 1) {
        all = peer(&mine, 0);
        for (int b = 1; b < blocks; ++b) all = join(all, peer(&mine, b));
    }
    const Ref ref(all.m);
    const float s = all.s, l2s = log2f(s);
    const bool empty = s == 0.f;
    const float lse = empty ? -INFINITY : ref.natural(l2s), ent = empty ? 0.f : (l2s - all.t / s) * LN2;
    if (rank == 0 && tid == 0) {
        if (a.lse) a.lse[row] = lse;
        if (a.entropy) a.entropy[row] = ent;
        if (a.logp) a.logp[row] = !scored ? 0.f : empty ? -INFINITY : ref.logp(at_y, l2s);
    }
    if (a.top && rank == 0) {
        // the blocks' lists, by rank among all of them
        const int n = a.top * blocks;
        for (int i = tid; i < n; i += LPT) cand[i] = blocks > 1 ? peer(best_of + i % a.top, i / a.top) : best_of[i];
        __syncthreads();
        for (int i = tid; i < n; i += LPT) {
            const uint64_t c = cand[i];
            int r = 0;
#pragma unroll 1
            for (int k = 0; k < n; ++k) r += cand[k] > c;
            if (c == 0 || r >= a.top) continue;          // 0: a place that a short part left free
            a.top_id[row * a.top + r] = int32_t(~uint32_t(c));
            a.top_logp[row * a.top + r] = empty ? -INFINITY : ref.logp(key_value(uint32_t(c >> 32)), l2s);
        }
    }
    if (GRAD) {
        const float gl = scored && !empty && a.glp ? a.glp[row] : 0.f, ge = a.gent ? a.gent[row] : 0.f;
        // g = -gl p - ge p (ln p + entropy), with ln p = (d - l2s) ln 2
        const float c0 = empty ? 0.f : fmaf(-ge, ent - l2s * LN2, -gl) / s, c1 = empty ? 0.f : -ge * LN2 / s;
        const Ragged<T> out(static_cast<T *>(a.dlogits) + row * a.ldd, a.V);
        const int hot = scored ? int(unsigned(y + x.shift) / N) - v0 : -1;
        uint4 *dst = reinterpret_cast<uint4 *>(out.p - x.shift) + v0;
        const bool same = out.shift == x.shift;          // whole vectors of one are whole vectors of the other
        auto grad = [&](uint4 raw) { return ref.far ? slope<T, true>(raw, ref, c0, c1) : slope<T, false>(raw, ref, c0, c1); };
        auto odd = [&](int i) {
            float v[N];
            Vec<T>::unpack(grad(fetch(i)), v);
            out.store(v0 + i, x.shift, v);
        };
        if (same) {
            int i = w0 + tid;
            for (; i + LPT < w1; i += 2 * LPT) {
                const uint4 r0 = __ldcs(src + i), r1 = __ldcs(src + i + LPT);
                __stcs(dst + i, grad(r0));
                __stcs(dst + i + LPT, grad(r1));
            }
            if (i < w1) __stcs(dst + i, grad(__ldcs(src + i)));
        } else {
            for (int i = w0 + tid; i < w1; i += LPT) odd(i);
        }
        if (end < nv) odd(end);
        // the target's own value, over what this thread stored for its vector
        if (hot >= 0 && hot < nv && tid == (hot == 0 && odd_first ? 0 : hot == nv - 1 && odd_last ? 1 : (hot - w0) % LPT)) {
            const float d = ref.far ? ref.at<true>(at_y) : ref.at<false>(at_y);
            out.p[y] = Vec<T>::put(fmaf(fast_exp2(d), fmaf(c1, fmaxf(d, -200.f), c0), gl));
        }
    }
    if (blocks > 1) meet(blocks);                        // no block leaves while another reads its statistics
}

// ---------------------------------------------------------------- clipping
// Bound by bytes: one read for the norm, one read and one write for the scaling.  Up to 1000
// tensors (their table travels as the kernel's parameters) take one cooperative launch: every block
// sums its chunks, the blocks meet, and each goes back over its chunks from the last one, whose
// values are still in L2.  More tensors take one launch a group for the norm and one for the
// scaling.  Measured: 220M bf16 values in one tensor 211 us (norm 71 us, 0.91 of the copy bandwidth;
// a copy of it takes 135 us), 100k values in 24 tensors 7 us.  220M values in 300 tensors: 226 us a
// call, 232 us in the first form with two launches.
constexpr int CT = 256;         // threads of a block
constexpr int CB = 4;           // blocks an SM
constexpr int CLIP_GRID = 152 * CB; // at most: as many as are resident together

template <int MAXS>
struct ClipSegs {
    int n, first_group;         // first_group: the total starts with this group of tensors
    float max_norm;
    int chunk;                  // 16-byte units of a chunk, a multiple of CT
    int64_t chunks;
    const void *src[MAXS];
    void *dst[MAXS];
    int64_t len[MAXS];
    int first[MAXS];            // a tensor's first chunk
    uint8_t bf16[MAXS];
};
struct ClipWs {                 // in the workspace
    unsigned *status, *ticket, *turn;
    float *part, *total;
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

// The part i0 .. i1 (16-byte units) of a tensor: its sum of squares, or its values times f.  Whole
// units eight at a time a thread; the ends of a tensor, and outputs aligned otherwise, value by value.
constexpr int CU = 8;
template <class T>
__device__ __forceinline__ float part_square(const void *src, int64_t n, int64_t i0, int64_t i1) {
    constexpr int N = Vec<T>::N;
    const Ragged<T> x(const_cast<T *>(static_cast<const T *>(src)), n);
    const uint4 *p = reinterpret_cast<const uint4 *>(x.p - x.shift);
    i1 = min(i1, x.vectors());
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    auto add = [&](uint4 raw) {
        float v[N];
        Vec<T>::unpack(raw, v);
#pragma unroll
        for (int e = 0; e < N; ++e) s[e & 3] = fmaf(v[e], v[e], s[e & 3]);
    };
    const int64_t w0 = i0 + !x.whole(i0), w1 = max(w0, i1 - !x.whole(i1 - 1));
    const int len = int(w1 - w0);
    p += w0;
    int i = threadIdx.x;
#pragma unroll 1
    for (; i + (CU - 1) * CT < len; i += CU * CT) {
        uint4 raw[CU];
#pragma unroll
        for (int u = 0; u < CU; ++u) raw[u] = __ldg(p + i + u * CT);
#pragma unroll
        for (int u = 0; u < CU; ++u) add(raw[u]);
    }
#pragma unroll 1
    for (; i < len; i += CT) add(__ldg(p + i));
    const int64_t end = threadIdx.x == 0 && w0 > i0 ? i0 : threadIdx.x == 1 && w1 < i1 && w1 >= w0 && i1 - 1 > i0 ? i1 - 1 : -1;
    if (end >= 0) {
        float v[N];
        x.load(end, v, 0.f);
#pragma unroll
        for (int e = 0; e < N; ++e) s[e & 3] = fmaf(v[e], v[e], s[e & 3]);
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

template <class T>
__device__ __forceinline__ void part_scale(const void *src, void *dst, int64_t n, int64_t i0, int64_t i1, float f) {
    constexpr int N = Vec<T>::N;
    const Ragged<T> x(const_cast<T *>(static_cast<const T *>(src)), n), y(static_cast<T *>(dst), n);
    const uint4 *p = reinterpret_cast<const uint4 *>(x.p - x.shift);
    uint4 *q = reinterpret_cast<uint4 *>(y.p - y.shift);
    i1 = min(i1, x.vectors());
    auto scaled = [&](uint4 raw) {
        float v[N];
        Vec<T>::unpack(raw, v);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] *= f;
        return Vec<T>::pack(v);
    };
    auto slowly = [&](int64_t i) {
        float v[N];
        x.load(i, v, 0.f);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] *= f;
        y.store(i, x.shift, v);
    };
    if (x.shift != y.shift) {
        for (int64_t i = i0 + threadIdx.x; i < i1; i += CT) slowly(i);
        return;
    }
    const int64_t w0 = i0 + !x.whole(i0), w1 = max(w0, i1 - !x.whole(i1 - 1));
    const int len = int(w1 - w0);
    p += w0;
    q += w0;
    // backwards: what was read last is read first
    int i = len - 1 - int(threadIdx.x);
#pragma unroll 1
    for (; i - (CU / 2 - 1) * CT >= 0; i -= CU / 2 * CT) {
        uint4 raw[CU / 2];
#pragma unroll
        for (int u = 0; u < CU / 2; ++u) raw[u] = __ldcs(p + i - u * CT);
#pragma unroll
        for (int u = 0; u < CU / 2; ++u) __stcs(q + i - u * CT, scaled(raw[u]));
    }
#pragma unroll 1
    for (; i >= 0; i -= CT) __stcs(q + i, scaled(__ldcs(p + i)));
    if (threadIdx.x == 0 && w0 > i0) slowly(i0);
    if (threadIdx.x == 1 && w1 < i1 && i1 - 1 > i0) slowly(i1 - 1);
}

// Sums over a block and over the blocks are plain fp32 trees of eight levels each, with up to two
// additions between them and one more a further group of tensors: 18 roundings, 1.1e-6 of the norm's
// square at worst.  (The fp64 pipe takes 2 us for them, as long as the rest of a small call.)  What a
// thread adds up of one tensor before that is plain fp32 too: four sums of 350 squares each for 220M
// values; the norms are within 2.1e-7 of the plain form's in the measured cases.
__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float r = red[threadIdx.x & (CT / 32 - 1)];
#pragma unroll
    for (int d = CT / 64; d; d >>= 1) r += __shfl_xor_sync(~0u, r, d);
    __syncthreads();
    return r;
}

// A block takes a contiguous range of chunks, so that it looks its tensor up once.
template <int MAXS>
__device__ __forceinline__ int64_t range(const ClipSegs<MAXS> &g, int64_t block) {
    return g.chunks * block / gridDim.x;
}

// The block's part of the sum of squares.  A thread's tensors add up as a sum and what its
// roundings lost: the fp64 pipe would take as long as the loads.
template <int MAXS>
__device__ __forceinline__ float sum_chunks(const ClipSegs<MAXS> &g) {
    float sum = 0.f, lost = 0.f;
    const int64_t c1 = range(g, int64_t(blockIdx.x) + 1);
    int64_t c = range(g, blockIdx.x);
    for (int s = seg_of(g, c); c < c1; ++s) {
        const int64_t next = s + 1 < g.n ? min(c1, int64_t(g.first[s + 1])) : c1;
        const int64_t i0 = (c - g.first[s]) * g.chunk, i1 = (next - g.first[s]) * g.chunk;
        const float x = g.bf16[s] ? part_square<__nv_bfloat16>(g.src[s], g.len[s], i0, i1)
                                  : part_square<float>(g.src[s], g.len[s], i0, i1);
        const float t = sum + x, y = t - sum, z = (sum - (t - y)) + (x - y);
        if (z == z) lost += z;                           // not where the sum is infinite
        sum = t;
        c = next;
    }
    return sum + lost;
}

// Hands in the block's sum; true in the last block to do so, which then has added all of them in the
// blocks' order and written the norm and the coefficient.
template <int MAXS>
__device__ __forceinline__ bool hand_in(const ClipSegs<MAXS> &g, float sum, const ClipWs &ws, float *out, float *red) {
    __shared__ bool last;
    sum = block_sum(sum, red);
    if (threadIdx.x == 0) {
        ws.part[blockIdx.x] = sum;
        __threadfence();
        last = atomicInc(ws.ticket, gridDim.x - 1) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return false;
    __threadfence();
    float v = 0.f;
    for (int b = threadIdx.x; b < int(gridDim.x); b += CT) v += __ldcg(ws.part + b);
    v = block_sum(v, red);
    if (threadIdx.x == 0) {
        if (!g.first_group) v += *ws.total;
        *ws.total = v;
        const float norm = sqrtf(v), c = g.max_norm / (norm + ADJ_CLIP_EPS);
        out[0] = norm;
        out[1] = c > 1.f ? 1.f : c;                      // NaN stays NaN
    }
    return true;
}

// The block's chunks, the last one first: its values were read last.
template <int MAXS>
__device__ __forceinline__ void scale_chunks(const ClipSegs<MAXS> &g, float f) {
    const int64_t c0 = range(g, blockIdx.x);
    int64_t c1 = range(g, int64_t(blockIdx.x) + 1);
    for (int s = seg_of(g, c1 - 1); c1 > c0; --s) {
        const int64_t c = max(c0, int64_t(g.first[s]));
        if (g.dst[s] && !(g.dst[s] == g.src[s] && f == 1.f)) {
            const int64_t i0 = (c - g.first[s]) * g.chunk, i1 = (c1 - g.first[s]) * g.chunk;
            if (g.bf16[s]) part_scale<__nv_bfloat16>(g.src[s], g.dst[s], g.len[s], i0, i1, f);
            else part_scale<float>(g.src[s], g.dst[s], g.len[s], i0, i1, f);
        }
        c1 = c;
    }
}

template <int MAXS>
__global__ __launch_bounds__(CT, CB) void k_clip_norm(const __grid_constant__ ClipSegs<MAXS> g, const ClipWs ws, float *out) {
    __shared__ float red[CT / 32];
    hand_in(g, sum_chunks(g), ws, out, red);
}
template <int MAXS>
__global__ __launch_bounds__(CT, CB) void k_clip_scale(const __grid_constant__ ClipSegs<MAXS> g, const float *out) {
    scale_chunks(g, out[1]);
}
// Both, with all blocks resident (cooperative launch).
template <int MAXS>
__global__ __launch_bounds__(CT, CB) void k_clip(const __grid_constant__ ClipSegs<MAXS> g, const ClipWs ws, float *out) {
    __shared__ float red[CT / 32];
    __shared__ float coef;
    __shared__ bool met;
    const unsigned turn = threadIdx.x == 0 ? ld_acquire(ws.turn) : 0u;     // before this block hands in
    const float sum = sum_chunks(g);
    const bool last = hand_in(g, sum, ws, out, red);
    if (threadIdx.x == 0) {
        met = true;
        if (last) {
            __threadfence();
            st_release(ws.turn, turn + 1);
        } else {
            int it = 0;
            while (ld_acquire(ws.turn) == turn && ++it < SPIN_LIMIT) {
            }
            if (it == SPIN_LIMIT) {                      // no coefficient: nothing is scaled, and the result says so
                record_timeout(ws.status);
                out[0] = out[1] = NAN;
                met = false;
            }
        }
        coef = __ldcg(out + 1);
    }
    __syncthreads();
    if (met) scale_chunks(g, coef);
}

// The next tensors from i on, as many as fit; returns where the next group starts.
template <int MAXS>
int64_t fill(ClipSegs<MAXS> &t, const adj_grad_seg *segs, int64_t i, int64_t nseg) {
    t.n = 0;
    t.chunks = 0;
    for (; i < nseg && t.n < MAXS; ++i) {
        if (segs[i].n == 0) continue;
        const bool bf = segs[i].dtype == ADJ_BF16;
        const int64_t bytes = (reinterpret_cast<uintptr_t>(segs[i].src) & 15u) + segs[i].n * (bf ? 2 : 4);
        const int64_t chunks = cdiv(bytes, 16 * int64_t(t.chunk));
        if (t.chunks + chunks >= (int64_t(1) << 31)) break;
        t.src[t.n] = segs[i].src;
        t.dst[t.n] = segs[i].dst;
        t.len[t.n] = segs[i].n;
        t.first[t.n] = int(t.chunks);
        t.bf16[t.n] = bf;
        t.chunks += chunks;
        ++t.n;
    }
    while (i < nseg && segs[i].n == 0) ++i;
    return i;
}

// Blocks that are resident together on the current device.
int clip_blocks() {
    static std::atomic<int> seen[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return CLIP_GRID;
    if (dev < 64 && (sms = seen[dev].load(std::memory_order_relaxed)) == 0) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) return CLIP_GRID;
        seen[dev].store(sms, std::memory_order_relaxed);
    }
    return sms > 0 ? std::min(CLIP_GRID, sms * CB) : CLIP_GRID;
}

template <int MAXS>
cudaError_t clip(const adj_grad_seg *segs, int64_t nseg, float max_norm, float *out, char *base, cudaStream_t st) {
    ClipWs ws;
    ws.status = reinterpret_cast<unsigned *>(base);
    ws.ticket = ws.status + 2;
    ws.turn = ws.status + 3;
    ws.part = reinterpret_cast<float *>(base + WS_HEADER);
    ws.total = ws.part + CLIP_GRID;
    ClipSegs<MAXS> t;
    t.max_norm = max_norm;
    t.first_group = 1;
    // chunks of 16 KB, four loads in flight a thread; of 4 KB where those would leave SMs idle
    int64_t bytes = 0;
    for (int64_t i = 0; i < nseg; ++i) bytes += segs[i].n * (segs[i].dtype == ADJ_BF16 ? 2 : 4);
    t.chunk = bytes < int64_t(152) * 16384 ? CT : 4 * CT;
    const int most = clip_blocks();
    auto grid = [&] { return unsigned(std::max<int64_t>(1, std::min<int64_t>(t.chunks, most))); };
    int64_t i = fill(t, segs, 0, nseg);
    if (i >= nseg) {
        ProfScope ps(K_CLIP_NORM, st);
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(grid());
        cfg.blockDim = dim3(CT);
        cfg.stream = st;
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeCooperative;
        at.val.cooperative = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, k_clip<MAXS>, t, ws, out);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    for (int pass = 0; pass < 2; ++pass)
        for (i = 0; i < nseg;) {
            i = fill(t, segs, i, nseg);
            ProfScope ps(pass ? K_CLIP_SCALE : K_CLIP_NORM, st);
            if (pass == 0) k_clip_norm<MAXS><<<grid(), CT, 0, st>>>(t, ws, out);
            else k_clip_scale<MAXS><<<grid(), CT, 0, st>>>(t, out);
            const cudaError_t e = cudaGetLastError();
            if (e != cudaSuccess) return e;
            t.first_group = 0;
        }
    return cudaSuccess;
}

}  // namespace

namespace {
template <class T, bool GRAD>
cudaError_t logprob(LogprobArgs a, cudaStream_t st) {
    const int64_t row = a.V * int64_t(sizeof(T)) + 16;
    a.blocks = 1;
    a.log_blocks = 0;
    // a row that the gradient reads again has to stay in L2 with the others in flight ...
    while (GRAD && a.blocks < 8 && row > a.blocks * ROW_PART) a.blocks = 1 << ++a.log_blocks;
    // ... and idle SMs are put to use while a part is at least one turn of the block's loads.  More
    // parts than that cost more than they even out (2048 x 50001 fp32: 86 us in one part, 128 in four).
    while (a.blocks < 8 && a.N * a.blocks * 2 <= 152 && row >= a.blocks * 2 * int64_t(LPU * LPT * 16)) a.blocks = 1 << ++a.log_blocks;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(a.N * a.blocks));
    cfg.blockDim = dim3(LPT);
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = unsigned(a.blocks);
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = a.blocks > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_logprob<T, GRAD>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}
}  // namespace

cudaError_t launch_logprob(const LogprobArgs &a, bool bf16, cudaStream_t st) {
    ProfScope ps(K_LOGPROB, st);
    if (bf16) return a.dlogits ? logprob<__nv_bfloat16, true>(a, st) : logprob<__nv_bfloat16, false>(a, st);
    return a.dlogits ? logprob<float, true>(a, st) : logprob<float, false>(a, st);
}

size_t clip_ws_bytes() { return WS_HEADER + (CLIP_GRID + 1) * sizeof(float); }

cudaError_t launch_grad_clip(const adj_grad_seg *segs, int64_t nseg, float max_norm, float *out, char *ws,
                             cudaStream_t st) {
    return nseg <= 64 ? clip<64>(segs, nseg, max_norm, out, ws, st) : clip<1000>(segs, nseg, max_norm, out, ws, st);
}

}  // namespace adj
