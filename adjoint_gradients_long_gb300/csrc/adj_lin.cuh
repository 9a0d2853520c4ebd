// adj_lin.cuh -- linear attention with a decay for each head: what its kernels share.
#pragma once
#include <atomic>

#include "adj_internal.cuh"

#define LIN_CUDA(x)                           \
    do {                                      \
        cudaError_t e_ = (x);                 \
        if (e_ != cudaSuccess) return e_;     \
    } while (0)

namespace adj {

inline int64_t lin_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
constexpr int LIN_CHUNK = 64, LIN_TC_CHUNK = 128;       // tokens of a chunk: fp32, bf16
inline int64_t lin_chunks(int64_t T, bool bf16) { return lin_div(T, bf16 ? LIN_TC_CHUNK : LIN_CHUNK); }

// The kernel's limit of dynamic shared memory, raised once a device (the call costs as much as a
// launch): to the most that any launch of it may ask for.
template <auto Kern>
cudaError_t allow_smem(size_t most = 232448 - 8192) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(most));
    if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// One call, sizes and arrays resolved on the host.
struct LinArgs {
    int64_t B, T, NC;           // NC chunks a sequence
    int H, Hk, Dk, Dv;
    int64_t ldq, ldk, ldv, ldo; // elements between tokens
    float scale;
    const void *q, *k, *v, *go;
    const float *g, *s0, *ds1;
    void *o, *dq, *dk, *dv;
    float *s1, *dg, *ds0;
    float *S, *dS;              // [B,H,NC,Dk,Dv]: the states entering / adjoint states leaving each chunk
    float *tot, *dtot;          // [B,H,NC]: the decay over each chunk (dtot: beside dS, where both are in flight)
    // bf16: S and dS of every chunk as sums of three bf16 instead; S, dS, tot are then those of segments.
    // The third parts lie in pieces of 32 columns, [B,H,NC] x [lin_pieces(Dv)][Dk][32]
    __nv_bfloat16 *shi, *slo, *s3, *zhi, *zlo, *z3;
    float *pq, *pk;             // Hk < H: dq, dk of every head [B,T,H,Dk] fp32, summed afterwards
};

__host__ __device__ constexpr int lin_pieces(int Dv) { return (Dv + 31) / 32; }

// exp(g) below this is under half the smallest fp32: the decay is zero, a new start.
constexpr float LIN_RESET = -104.f;

// A sum kept as hi + lo, 48 bits: the fp64 pipe is too slow for one warp to keep up with a chunk.
struct Sum2 {
    float hi, lo;
    __device__ __forceinline__ static Sum2 two(float a, float b) {      // a + b exactly
        const float s = a + b, t = s - a;
        return Sum2{s, (a - (s - t)) + (b - t)};
    }
    __device__ __forceinline__ static Sum2 log2_of(float x) {           // x log2 e
        constexpr float H = 1.44269502162933349609375f, L = 1.925963033500011079e-8f;
        const float p = x * H;
        return Sum2{p, fmaf(x, L, fmaf(x, H, -p))};
    }
    __device__ __forceinline__ Sum2 operator+(Sum2 o) const {
        const Sum2 s = two(hi, o.hi);
        const float l = s.lo + (lo + o.lo), h = s.hi + l;
        return Sum2{h, l - (h - s.hi)};
    }
    __device__ __forceinline__ Sum2 operator-(Sum2 o) const { return *this + Sum2{-o.hi, -o.lo}; }
    __device__ __forceinline__ float value() const { return hi + lo; }
    __device__ __forceinline__ Sum2 up(int d) const { return Sum2{__shfl_up_sync(~0u, hi, d), __shfl_up_sync(~0u, lo, d)}; }
    __device__ __forceinline__ Sum2 from(int l) const { return Sum2{__shfl_sync(~0u, hi, l), __shfl_sync(~0u, lo, l)}; }
};

// The decays of one chunk.  With g_t the tokens' log decays in powers of two, G_t their
// inclusive sum from the chunk's start and r_t the number of new starts up to t, the decay
// from token j to token i >= j is 2^(G_i - G_j) where r_i = r_j, and zero otherwise.  G is kept
// as a pair hi + lo, so that a difference of two long sums is as exact as a short sum.
template <int C>
struct LinDecay {
    float hi[C], lo[C];
    int r[C];

    // from token j to token i; j <= i
    __device__ __forceinline__ float pair(int i, int j) const {
        return r[i] == r[j] ? fast_exp2((hi[i] - hi[j]) + (lo[i] - lo[j])) : 0.f;
    }
    // from before the chunk to token i, from token j to the chunk's end
    __device__ __forceinline__ float first(int i) const { return r[i] == 0 ? fast_exp2(hi[i] + lo[i]) : 0.f; }
    __device__ __forceinline__ float last(int j) const { return pair(C - 1, j); }
    __device__ __forceinline__ float total() const { return first(C - 1); }

    // by one whole warp: g[n * pitch], n < len (tokens past len have decay 1)
    __device__ void fill(const float *g, int64_t pitch, int len) {
        const int lane = threadIdx.x & 31;
        constexpr int PER = C / 32;
        Sum2 s[PER], sum{0.f, 0.f};
        int c[PER], cnt = 0;
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int t = lane * PER + u;
            const float x = t < len ? __ldg(g + t * pitch) : 0.f;
            const bool cut = x < LIN_RESET;
            sum = sum + Sum2::log2_of(cut ? 0.f : x);
            cnt += cut;
            s[u] = sum;
            c[u] = cnt;
        }
        Sum2 run = sum;
        int rc = cnt;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const Sum2 a = run.up(d);
            const int b = __shfl_up_sync(~0u, rc, d);
            if (lane >= d) {
                run = a + run;
                rc += b;
            }
        }
        Sum2 before = run.up(1);
        if (lane == 0) before = Sum2{0.f, 0.f};
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const Sum2 G = before + s[u];
            const int t = lane * PER + u;
            hi[t] = G.hi;
            lo[t] = G.lo;
            r[t] = rc - cnt + c[u];
        }
    }
};

// bytes of workspace after the header, and the arrays in it
size_t lin_ws_bytes(const LinArgs &a, bool bwd, bool bf16);
void lin_ws_carve(LinArgs &a, bool bwd, bool bf16, void *base);

cudaError_t launch_lin_fwd(const LinArgs &a, bool bf16, unsigned *status, cudaStream_t st);
cudaError_t launch_lin_bwd(const LinArgs &a, bool bf16, unsigned *status, cudaStream_t st);
// The tensor-core forward pass (bf16 storage), and how it cuts a head's tokens: nseg segments of
// cps chunks.  Its states are those of the segments: S [B,H,nseg,Dk,Dv], tot [B,H,nseg].
struct LinSplit {
    int nseg, cps;
};
LinSplit lin_split(const LinArgs &a, bool bwd);
cudaError_t launch_lin_tc_fwd(const LinArgs &a, unsigned *status, cudaStream_t st);
// the tensor-core backward pass but for the sum over shared heads
cudaError_t launch_lin_tc_bwd(const LinArgs &a, unsigned *status, cudaStream_t st);
// Every entry of S [B,H,n,Dk,Dv] becomes the state before it (dirs & 1), every entry of dS the
// adjoint state after it (dirs & 2).
cudaError_t launch_lin_scan(const LinArgs &a, int64_t n, int dirs, cudaStream_t st);
cudaError_t launch_lin_step(const LinArgs &a, bool bf16, float *state, int64_t n_slots, const int32_t *slots,
                            cudaStream_t st);

}  // namespace adj
