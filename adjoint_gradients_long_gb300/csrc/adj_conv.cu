// adj_conv.cu -- the short causal convolution of a selective layer: prompts, gradients and single
// tokens.  include/adj.h defines it.
//
// A thread walks a run of consecutive tokens for four channels, with the last W-1 inputs, the weights and
// the sums of a token in registers, so each value is read once (and W-1 of them again by the run
// after it, mostly from L2) and written once.  Bound by HBM: the arithmetic is W multiply-adds and
// one sigmoid a value.  Four channels, not eight: eight took 162 registers forwards and 255 backwards,
// too few warps to cover HBM's latency.  With W = 4 the gradients still spill (60 bytes stored and 164 loaded
// a thread in bf16, 80 and 160 in fp32), and so do the outputs in fp32 (52 and 68).  Measured: 32768 tokens x
// 2048 channels bf16 50 us (0.80 of the copy bandwidth), fp32 96 (0.83); gradients of 16384 tokens bf16 54 us
// (0.55), fp32 78 (0.76).  A block holds VG quads of channels side by side and
// 256 / VG runs, VG the power of two that covers the channels, 64 at most: neighbouring threads
// read neighbouring quads.
//
// Gradient: with dp_t = go_t act'(p_t),
//     dc_i = sum_j w_j dp_{i-j},    dw_j = sum_t dp_t c_{t+j},
// the walk goes forward and emits dx of a token once dp of the W-1 tokens after it are known.  A run
// reads W-1 tokens beyond its end for that, and never beyond its sequence's.
#include "adj_profile.cuh"
#include "adj_seq.cuh"

namespace adj {
namespace {

constexpr int CT = 256;         // threads of a block
// A thread's next tokens, on their way to its own places in shared memory, 32 KB a block: as many in registers
// would leave too few warps.  It waits for its own copies alone.
template <class T, int ARRAYS>
struct Ring {
    static constexpr int TOKENS = int(32768 / (CT * sizeof(Raw4<T>) * ARRAYS));     // a power of two
    Raw4<T> v[TOKENS][ARRAYS][CT];
    __device__ __forceinline__ Raw4<T> get(int i, int array) const { return v[i & (TOKENS - 1)][array][threadIdx.x]; }
    __device__ __forceinline__ void start(int i, int array, const T *p) {
        const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(&v[i & (TOKENS - 1)][array][threadIdx.x]));
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(p), "n"(sizeof(Raw4<T>)) : "memory");
    }
    __device__ __forceinline__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    template <int N>
    __device__ __forceinline__ static void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
};

template <class T>
__device__ __forceinline__ const T *row(const void *p, int64_t i, int64_t ld, int c) {
    return static_cast<const T *>(p) + i * ld + c;
}

using adj::operator+;                   // beside those of Four
using adj::sigmoid4;

// Four channels as two packed pairs: a multiply-add takes half the instructions
struct Four {
    pair_t a, b;
    __device__ __forceinline__ Four() {}
    __device__ __forceinline__ explicit Four(float x) : a(pk(x, x)), b(a) {}
    __device__ __forceinline__ explicit Four(float4 v) : a(pk(v.x, v.y)), b(pk(v.z, v.w)) {}
    __device__ __forceinline__ Four(pair_t a_, pair_t b_) : a(a_), b(b_) {}
    __device__ __forceinline__ float4 get() const {
        float4 v;
        upk(a, v.x, v.y);
        upk(b, v.z, v.w);
        return v;
    }
};
__device__ __forceinline__ Four operator*(Four x, Four y) { return Four(mul2(x.a, y.a), mul2(x.b, y.b)); }
__device__ __forceinline__ Four operator+(Four x, Four y) { return Four(add2(x.a, y.a), add2(x.b, y.b)); }
__device__ __forceinline__ Four fma4(Four x, Four y, Four z) { return Four(fma2(x.a, y.a, z.a), fma2(x.b, y.b, z.b)); }
__device__ __forceinline__ Four sigmoid4(Four x) { return Four(sigmoid4(x.get())); }

// Weights and bias of four channels; w is [P][W], so theirs are W vectors in a row
template <int W>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int c, Four (&w)[W], Four &bias) {
    union {
        float4 v[W];
        float f[4 * W];
    } u;
#pragma unroll
    for (int j = 0; j < W; ++j) u.v[j] = __ldg(reinterpret_cast<const float4 *>(a.w + int64_t(c) * W) + j);
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = Four(make_float4(u.f[j], u.f[W + j], u.f[2 * W + j], u.f[3 * W + j]));
    bias = Four(a.bias ? __ldg(reinterpret_cast<const float4 *>(a.bias + c)) : f4(0.f));
}

// Entry i of sequence b's list (its state, then its tokens from `begin` on)
template <class T, int W>
__device__ __forceinline__ Raw4<T> entry(const ConvArgs &a, int64_t b, int64_t begin, int64_t i, int c) {
    Raw4<T> r;
    if (i >= W - 1) r.load(row<T>(a.x, begin + i - (W - 1), a.ldx, c));
    else if (a.s0) r.load(row<T>(a.s0, b * (W - 1) + i, a.P, c));
    else r.zero();
    return r;
}

// Offsets of up to 256 sequences, read by the block together: the search for a run's sequence then waits for
// shared memory, not five times for L2.  (All threads of the block.)
constexpr int NEAR = 256;
__device__ __forceinline__ Seqs near(const Seqs &q, int64_t *offs) {
    Seqs n = q;
    if (q.off && q.B <= NEAR) {
        for (int i = threadIdx.x; i <= int(q.B); i += CT) offs[i] = q.off[i];
        __syncthreads();
        n.off = offs;
    }
    return n;
}

struct Place {
    int c;                      // first of the thread's four channels
    int run;                    // of the block's runs
    bool in;
    __device__ Place(int vg, int P) {
        const int v = int(blockIdx.y) * vg + int(threadIdx.x) % vg;
        run = int(threadIdx.x) / vg;
        c = v * 4;
        in = c < P;
    }
};

// Blocks below `runs` take tokens, those above write the states after the last tokens.
template <class T, int W>
__global__ __launch_bounds__(CT, 4) void k_conv_fwd(const ConvArgs a, int vg, int tr, int64_t runs) {
    typedef Ring<T, 1> R;
    __shared__ R ring;
    __shared__ int64_t offs[NEAR + 1];
    const Seqs q = near(a.q, offs);
    const Place at(vg, a.P);
    if (!at.in) return;
    const int c = at.c, rg = CT / vg;
    if (int64_t(blockIdx.x) >= runs) {
        const int64_t b = (blockIdx.x - runs) * rg + at.run;
        if (b >= q.B) return;
        const int64_t begin = q.begin(b), n = max(int64_t(0), q.end(b) - begin);
        for (int i = 0; i < W - 1; ++i)
            entry<T, W>(a, b, begin, n + i, c).store(static_cast<T *>(a.s1) + (b * (W - 1) + i) * a.P + c);
        return;
    }
    int64_t t = (int64_t(blockIdx.x) * rg + at.run) * tr;
    const int64_t stop = min(t + tr, q.rows);
    if (t >= stop) return;
    Four w[W], bias, x[W];
    load_taps<W>(a, c, w, bias);
    if (q.off) t = max(t, q.at(0));
    while (t < stop) {
        const int64_t b = q.find(t);
        if (b < 0) return;
        const int64_t begin = q.begin(b), end = min(q.end(b), stop);
        // x[1..W-1]: the W-1 entries before token t
#pragma unroll
        for (int j = 0; j < W - 1; ++j) x[j + 1] = Four(entry<T, W>(a, b, begin, t - begin + j, c).get());
        // pointers and counts inside the run: 64-bit comparisons a token cost more than its arithmetic
        const T *px = row<T>(a.x, t, a.ldx, c);
        T *py = static_cast<T *>(a.y) + t * a.ldy + c;
        const int n = int(end - t);
        constexpr int FU = 4, AHEAD = R::TOKENS / FU - 1;
        auto fetch = [&](int i) {
#pragma unroll
            for (int u = 0; u < FU; ++u)
                if (i + u < n) ring.start(i + u, 0, px + u * a.ldx);
            px += FU * a.ldx;
            ring.commit();
        };
#pragma unroll
        for (int g = 0; g < AHEAD; ++g) fetch(g * FU);
        auto token = [&](const Raw4<T> &in) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) x[j] = x[j + 1];
            x[W - 1] = Four(in.get());
            Four p = bias;
#pragma unroll
            for (int j = 0; j < W; ++j) p = fma4(w[j], x[j], p);
            st4(py, (a.act ? p * sigmoid4(p) : p).get());
            py += a.ldy;
        };
        for (int i = 0; i < n; i += FU) {
            fetch(i + AHEAD * FU);
            ring.template wait<AHEAD>();
            Raw4<T> now[FU];
#pragma unroll
            for (int u = 0; u < FU; ++u) now[u] = ring.get(i + u, 0);
            if (i + FU <= n) {                                      // straight on: the window moves by names alone
#pragma unroll
                for (int u = 0; u < FU; ++u) token(now[u]);
            } else {
#pragma unroll
                for (int u = 0; u < FU; ++u)
                    if (i + u < n) token(now[u]);
            }
        }
        t = end;
    }
}

// Blocks below `runs` take tokens, those above write ds0.
template <class T, int W>
__global__ __launch_bounds__(CT, 2) void k_conv_bwd(const ConvArgs a, int vg, int tr, int64_t runs) {
    typedef Ring<T, 2> R;
    __shared__ R ring;
    __shared__ float4 sum[CT];
    __shared__ int64_t offs[NEAR + 1];
    const Seqs q = near(a.q, offs);
    const Place at(vg, a.P);
    const int c = at.c, rg = CT / vg;
    Four w[W], bias, x[W], dp[W], dw[W], db(0.f);
    if (at.in) load_taps<W>(a, c, w, bias);
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j] = dp[j] = Four(0.f);
    // one token: its entry joins x[W-1], the cotangent of its sum dp[W-1]
    auto token = [&](const Raw4<T> &in, const Raw4<T> &cot) {
        x[W - 1] = Four(in.get());
        Four g(cot.get());
        if (a.act) {
            Four p = bias;
#pragma unroll
            for (int j = 0; j < W; ++j) p = fma4(w[j], x[j], p);
            // s (1 + p (1 - s)) = s + (p s) (1 - s)
            const Four s = sigmoid4(p);
            g = g * fma4(p * s, fma4(s, Four(-1.f), Four(1.f)), s);
        }
        dp[W - 1] = g;
    };
    auto shift = [&]() {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            x[j] = x[j + 1];
            dp[j] = dp[j + 1];
        }
    };
    auto sum_up = [&]() {
        db = db + dp[W - 1];
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j] = fma4(dp[W - 1], x[j], dw[j]);
    };
    if (int64_t(blockIdx.x) >= runs) {
        // dc of the entries of the state: from the first W-1 tokens, and from ds1 where a sequence is shorter
        const int64_t b = (blockIdx.x - runs) * rg + at.run;
        if (!at.in || b >= q.B) return;
        const int64_t begin = q.begin(b), n = max(int64_t(0), q.end(b) - begin);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) x[j + 1] = Four(entry<T, W>(a, b, begin, j, c).get());
        Four ds[W - 1];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            Raw4<T> r;
            r.zero();
            if (a.ds1 && i >= n) r.load(row<T>(a.ds1, b * (W - 1) + (i - n), a.P, c));
            ds[i] = Four(r.get());
        }
#pragma unroll
        for (int t = 0; t < W - 1; ++t) {
            if (t >= n) break;
            shift();
            Raw4<T> in, cot;
            in.load(row<T>(a.x, begin + t, a.ldx, c));
            cot.load(row<T>(a.go, begin + t, a.ldy, c));
            token(in, cot);
#pragma unroll
            for (int j = 0; j < W - 1 - t; ++j) ds[t + j] = fma4(w[j], dp[W - 1], ds[t + j]);
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i) st4(static_cast<T *>(a.ds0) + (b * (W - 1) + i) * a.P + c, ds[i].get());
        return;
    }
    int64_t t = (int64_t(blockIdx.x) * rg + at.run) * tr;
    const int64_t stop = at.in ? min(t + tr, q.rows) : 0;
    if (q.off && t < stop) t = max(t, q.at(0));
    while (t < stop) {
        const int64_t b = q.find(t);
        if (b < 0) break;
        const int64_t begin = q.begin(b), end = q.end(b), last = min(end, stop), until = last + W - 1;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            x[j + 1] = Four(entry<T, W>(a, b, begin, t - begin + j, c).get());
            dp[j + 1] = Four(0.f);
        }
        const T *px = row<T>(a.x, t, a.ldx, c), *pg = row<T>(a.go, t, a.ldy, c);
        T *pd = static_cast<T *>(a.dx) + t * a.ldx + c;
        // counted from the first token here: tokens that exist, that this run sums up and emits, that it walks
        const int left = int(min(end - t, int64_t(tr + W))), own = int(last - t), all = int(until - t);
        const int64_t tail = end - (W - 1) - t;                     // the first token that s1 holds
        constexpr int CU = R::TOKENS / 2, AHEAD = R::TOKENS / CU - 1;
        auto fetch = [&](int i) {
#pragma unroll
            for (int u = 0; u < CU; ++u)
                if (i + u < left && i + u < all) {
                    ring.start(i + u, 0, px + u * a.ldx);
                    ring.start(i + u, 1, pg + u * a.ldy);
                }
            px += CU * a.ldx;
            pg += CU * a.ldy;
            ring.commit();
        };
#pragma unroll
        for (int g = 0; g < AHEAD; ++g) fetch(g * CU);
        for (int i = 0; i < all; i += CU) {
            fetch(i + AHEAD * CU);
            ring.template wait<AHEAD>();
            Raw4<T> cx[CU], cg[CU];
#pragma unroll
            for (int u = 0; u < CU; ++u) {
                cx[u] = ring.get(i + u, 0);
                cg[u] = ring.get(i + u, 1);
            }
            // dx of the token W-1 behind: complete now
            auto emit = [&](Four d) {
#pragma unroll
                for (int j = 0; j < W; ++j) d = fma4(w[W - 1 - j], dp[j], d);
                st4(pd, d.get());
                pd += a.ldx;
            };
            if (i >= W - 1 && i + CU <= own && !(a.ds1 && i + CU - W >= tail)) {
                // straight on: the windows move by names alone
#pragma unroll
                for (int u = 0; u < CU; ++u) {
                    shift();
                    token(cx[u], cg[u]);
                    sum_up();
                    emit(Four(0.f));
                }
            } else {
#pragma unroll
                for (int u = 0; u < CU; ++u) {
                    const int k = i + u, s = k - (W - 1);
                    if (k >= all) break;
                    shift();
                    if (k < left) token(cx[u], cg[u]);
                    else dp[W - 1] = Four(0.f);
                    if (k < own) sum_up();
                    if (s >= 0) {
                        Four d(0.f);
                        if (a.ds1 && s >= tail) {
                            Raw4<T> r;
                            r.load(row<T>(a.ds1, b * (W - 1) + (s - tail), a.P, c));
                            d = Four(r.get());
                        }
                        emit(d);
                    }
                }
            }
        }
        t = last;
    }
    // the block's sums over its runs, in their order
#pragma unroll
    for (int k = 0; k <= W; ++k) {
        __syncthreads();
        sum[threadIdx.x] = (k < W ? dw[k < W ? k : 0] : db).get();  // thread = run vg + quad
        __syncthreads();
        const int p = (int(blockIdx.y) * vg + int(threadIdx.x)) * 4;
        if (int(threadIdx.x) < vg && p < a.P) {
            float4 v = f4(0.f);
            for (int r = 0; r < rg; ++r) v = v + sum[r * vg + threadIdx.x];
            *reinterpret_cast<float4 *>(a.part + (int64_t(blockIdx.x) * (W + 1) + k) * a.P + p) = v;
        }
    }
}

// dw [P][W] and dbias from the blocks' sums, in their order
__global__ __launch_bounds__(CT) void k_conv_join(const ConvArgs a, int64_t blocks) {
    const int64_t i = int64_t(blockIdx.x) * CT + threadIdx.x, n = int64_t(a.W + 1) * a.P;
    if (i >= n) return;
    const int k = int(i / a.P), p = int(i - int64_t(k) * a.P);
    float s = 0.f;
#pragma unroll 16
    for (int64_t b = 0; b < blocks; ++b) s += __ldg(a.part + b * n + i);
    if (k < a.W) a.dw[int64_t(p) * a.W + k] = s;
    else if (a.dbias) a.dbias[p] = s;
}

template <class T, int W>
__global__ __launch_bounds__(CT) void k_conv_step(const ConvArgs a, T *state, int64_t n_slots, const int32_t *slots) {
    const int pv = a.P / 4;
    const int64_t i = int64_t(blockIdx.x) * CT + threadIdx.x, b = i / pv;
    if (b >= a.q.B) return;
    const int c = int(i - b * pv) * 4;
    const int64_t slot = slots ? int64_t(__ldg(slots + b)) : b;
    T *y = static_cast<T *>(a.y) + b * a.ldy + c;
    if (slot < 0 || slot >= n_slots) {
        st4(y, f4(0.f));
        return;
    }
    Raw4<T> r[W];
    T *s = state + slot * (W - 1) * a.P + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) r[j].load_own(s + int64_t(j) * a.P);
    r[W - 1].load(row<T>(a.x, b, a.ldx, c));
    Four w[W], p;
    load_taps<W>(a, c, w, p);
#pragma unroll
    for (int j = 0; j < W; ++j) p = fma4(w[j], Four(r[j].get()), p);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) r[j + 1].store(s + int64_t(j) * a.P);
    st4(y, (a.act ? p * sigmoid4(p) : p).get());
}

// quads side by side in a block, runs of `tr` tokens, blocks of runs
struct ConvGrid {
    int vg, tr;
    int64_t runs;
};
// The longest runs (the fewest tokens read twice) of which there are still `want` threads' worth for
// the loads in flight to cover HBM's latency.  Measured with 2048 channels, bf16, us (tokens: as it is; half of `want`;
// twice): outputs 16384: 27.9; 28.6; 31.8, 4096: 9.9; 9.2; 13.7.  Gradients 16384: 54.7; 54.7; 65.3, 4096: 20.9; 20.2;
// 27.3.  Half the longest run: outputs 32768 50.0 against 48.2, gradients 16384 65.2 against 54.7; twice: the same, but
// gradients 32768 97 against 108.  Twice the shortest: outputs 77 3.9 against 3.4, gradients 512 12.4 against 9.9; half
// (gradients): 11.4 against 9.9.
ConvGrid conv_grid(const ConvArgs &a, int longest, int shortest, int64_t want) {
    const int pv = a.P / 4;
    ConvGrid g{1, longest, 0};
    while (g.vg < pv && g.vg < 64) g.vg *= 2;
    while (g.tr > shortest && seq_div(a.q.rows, g.tr) * pv < want) g.tr /= 2;
    g.runs = seq_div(a.q.rows, int64_t(g.tr) * (CT / g.vg));
    return g;
}
ConvGrid fwd_grid(const ConvArgs &a) { return conv_grid(a, 64, 4, 152 * 1024); }
ConvGrid bwd_grid(const ConvArgs &a) { return conv_grid(a, 128, 8, 152 * 384); }

// f(type, taps) for the call's type and taps
template <class F>
void pick(const ConvArgs &a, bool bf16, F f) {
    using std::integral_constant;
    auto taps = [&](auto type) {
        if (a.W == 2) f(type, integral_constant<int, 2>());
        else if (a.W == 3) f(type, integral_constant<int, 3>());
        else f(type, integral_constant<int, 4>());
    };
    if (bf16) taps(__nv_bfloat16());
    else taps(0.f);
}

}  // namespace

size_t conv_ws_bytes(const ConvArgs &a) { return size_t(bwd_grid(a).runs) * (a.W + 1) * a.P * sizeof(float); }

cudaError_t launch_conv_fwd(const ConvArgs &a, bool bf16, cudaStream_t st) {
    const ConvGrid g = fwd_grid(a);
    const int64_t blocks = g.runs + (a.s1 ? seq_div(a.q.B, CT / g.vg) : 0);
    if (blocks == 0) return cudaSuccess;
    const dim3 grid(unsigned(blocks), unsigned(seq_div(a.P / 4, g.vg)));
    ProfScope p(K_CONV_FWD, st);
    pick(a, bf16, [&](auto t, auto w) { k_conv_fwd<decltype(t), decltype(w)::value><<<grid, CT, 0, st>>>(a, g.vg, g.tr, g.runs); });
    return cudaGetLastError();
}

cudaError_t launch_conv_bwd(const ConvArgs &a, bool bf16, cudaStream_t st) {
    const ConvGrid g = bwd_grid(a);
    const int64_t blocks = g.runs + (a.ds0 ? seq_div(a.q.B, CT / g.vg) : 0);
    if (blocks) {
        const dim3 grid(unsigned(blocks), unsigned(seq_div(a.P / 4, g.vg)));
        ProfScope p(K_CONV_BWD, st);
        pick(a, bf16, [&](auto t, auto w) { k_conv_bwd<decltype(t), decltype(w)::value><<<grid, CT, 0, st>>>(a, g.vg, g.tr, g.runs); });
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    ProfScope p(K_CONV_BWD, st);
    k_conv_join<<<unsigned(seq_div(int64_t(a.W + 1) * a.P, CT)), CT, 0, st>>>(a, g.runs);
    return cudaGetLastError();
}

cudaError_t launch_conv_step(const ConvArgs &a, bool bf16, void *state, int64_t n_slots, const int32_t *slots,
                             cudaStream_t st) {
    const unsigned blocks = unsigned(seq_div(a.q.B * (a.P / 4), CT));
    ProfScope p(K_CONV_STEP, st);
    pick(a, bf16, [&](auto t, auto w) {
        typedef decltype(t) T;
        k_conv_step<T, decltype(w)::value><<<blocks, CT, 0, st>>>(a, static_cast<T *>(state), n_slots, slots);
    });
    return cudaGetLastError();
}

}  // namespace adj
