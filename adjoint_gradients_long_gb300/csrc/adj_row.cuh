// adj_row.cuh -- rows of logits: vectors of 16 bytes at any alignment, values in order, and the blocks
// of a cluster that share a row.
#pragma once
#include "adj_internal.cuh"

namespace adj {

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

// Order of the top list as unsigned integers: NaN above +inf, the zeros equal.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return k == 0xFFFFFFFFu ? NAN : __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// ---------------------------------------------------------------- blocks of a cluster
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

}  // namespace adj
