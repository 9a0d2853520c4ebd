// adj_conv.cu -- the short causal convolution of a selective layer: prompts, gradients and single
// tokens.  include/adj.h defines it.
//
// A thread walks a run of consecutive tokens for eight channels (16 bytes of bf16), with the last W-1
// inputs, the weights and the sums of a token in registers, so each value is read once (and W-1 of
// them again by the run after it, mostly from L2) and written once.  Bound by HBM: the arithmetic is
// W multiply-adds and one sigmoid a value.  A block holds VG vectors of channels side by side and
// 256 / VG runs, VG the power of two that covers the channels, 32 at most: neighbouring threads
// read neighbouring vectors.
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
constexpr int CU = 4;           // tokens in flight a thread

template <class T>
__device__ __forceinline__ const T *row(const void *p, int64_t i, int64_t ld, int c) {
    return static_cast<const T *>(p) + i * ld + c;
}

// weights [W][8] and bias of eight channels; w is [P][W]
template <int W>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int c, float (&w)[W][8], float (&bias)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = __ldg(a.w + int64_t(c + e) * W + j);
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[e] = a.bias ? __ldg(a.bias + c + e) : 0.f;
}

// Entry i of sequence b's list (its state, then its tokens from `begin` on)
template <class T, int W>
__device__ __forceinline__ Raw8<T> entry(const ConvArgs &a, int64_t b, int64_t begin, int64_t i, int c) {
    Raw8<T> r;
    if (i >= W - 1) r.load(row<T>(a.x, begin + i - (W - 1), a.ldx, c));
    else if (a.s0) r.load(row<T>(a.s0, b * (W - 1) + i, a.P, c));
    else r.zero();
    return r;
}

struct Place {
    int c;                      // first of the thread's eight channels
    int run;                    // of the block's runs
    bool in;
    __device__ Place(int vg, int P) {
        const int v = int(blockIdx.y) * vg + int(threadIdx.x) % vg;
        run = int(threadIdx.x) / vg;
        c = v * 8;
        in = c < P;
    }
};

// Blocks below `runs` take tokens, those above write the states after the last tokens.
template <class T, int W>
__global__ __launch_bounds__(CT) void k_conv_fwd(const ConvArgs a, int vg, int tr, int64_t runs) {
    const Place at(vg, a.P);
    if (!at.in) return;
    const int c = at.c, rg = CT / vg;
    if (int64_t(blockIdx.x) >= runs) {
        const int64_t b = (blockIdx.x - runs) * rg + at.run;
        if (b >= a.q.B) return;
        const int64_t begin = a.q.begin(b), n = max(int64_t(0), a.q.end(b) - begin);
        for (int i = 0; i < W - 1; ++i)
            entry<T, W>(a, b, begin, n + i, c).store(static_cast<T *>(a.s1) + (b * (W - 1) + i) * a.P + c);
        return;
    }
    int64_t t = (int64_t(blockIdx.x) * rg + at.run) * tr;
    const int64_t stop = min(t + tr, a.q.rows);
    if (t >= stop) return;
    float w[W][8], bias[8], x[W][8];
    load_taps<W>(a, c, w, bias);
    if (a.q.off) t = max(t, a.q.at(0));
    while (t < stop) {
        const int64_t b = a.q.find(t);
        if (b < 0) return;
        const int64_t begin = a.q.begin(b), end = min(a.q.end(b), stop);
        // x[1..W-1]: the W-1 entries before token t
#pragma unroll
        for (int j = 0; j < W - 1; ++j) entry<T, W>(a, b, begin, t - begin + j, c).get(x[j + 1]);
        Raw8<T> next[CU];
#pragma unroll
        for (int u = 0; u < CU; ++u)
            if (t + u < end) next[u].load(row<T>(a.x, t + u, a.ldx, c));
        for (; t < end; t += CU) {
            Raw8<T> now[CU];
#pragma unroll
            for (int u = 0; u < CU; ++u) now[u] = next[u];
#pragma unroll
            for (int u = 0; u < CU; ++u)
                if (t + CU + u < end) next[u].load(row<T>(a.x, t + CU + u, a.ldx, c));
#pragma unroll
            for (int u = 0; u < CU; ++u) {
                if (t + u >= end) break;
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) x[j][e] = x[j + 1][e];
                }
                now[u].get(x[W - 1]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float p = bias[e];
#pragma unroll
                    for (int j = 0; j < W; ++j) p = fmaf(w[j][e], x[j][e], p);
                    y[e] = a.act ? p * sigmoid_f(p) : p;
                }
                Raw8<T>::of(y).store(static_cast<T *>(a.y) + (t + u) * a.ldy + c);
            }
        }
        t = end;
    }
}

// Blocks below `runs` take tokens, those above write ds0.
template <class T, int W>
__global__ __launch_bounds__(CT) void k_conv_bwd(const ConvArgs a, int vg, int tr, int64_t runs) {
    __shared__ float sum[CT * 8];
    const Place at(vg, a.P);
    const int c = at.c, rg = CT / vg;
    float w[W][8], bias[8], x[W][8], dp[W][8], dw[W][8], db[8];
    if (at.in) load_taps<W>(a, c, w, bias);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        db[e] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][e] = dp[j][e] = 0.f;
    }
    // one token: its entry joins x[W-1], the cotangent of its sum dp[W-1]
    auto token = [&](const Raw8<T> &in, const Raw8<T> &cot) {
        float g[8];
        in.get(x[W - 1]);
        cot.get(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (a.act) {
                float p = bias[e];
#pragma unroll
                for (int j = 0; j < W; ++j) p = fmaf(w[j][e], x[j][e], p);
                const float s = sigmoid_f(p);
                g[e] *= s * fmaf(p, 1.f - s, 1.f);
            }
            dp[W - 1][e] = g[e];
        }
    };
    auto shift = [&]() {
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                x[j][e] = x[j + 1][e];
                dp[j][e] = dp[j + 1][e];
            }
    };
    if (int64_t(blockIdx.x) >= runs) {
        // dc of the entries of the state: from the first W-1 tokens, and from ds1 where a sequence is shorter
        const int64_t b = (blockIdx.x - runs) * rg + at.run;
        if (!at.in || b >= a.q.B) return;
        const int64_t begin = a.q.begin(b), n = max(int64_t(0), a.q.end(b) - begin);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) entry<T, W>(a, b, begin, j, c).get(x[j + 1]);
        float ds[W - 1][8];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            Raw8<T> r;
            r.zero();
            if (a.ds1 && i >= n) r.load(row<T>(a.ds1, b * (W - 1) + (i - n), a.P, c));
            r.get(ds[i]);
        }
#pragma unroll
        for (int t = 0; t < W - 1; ++t) {
            if (t >= n) break;
            shift();
            Raw8<T> in, cot;
            in.load(row<T>(a.x, begin + t, a.ldx, c));
            cot.load(row<T>(a.go, begin + t, a.ldy, c));
            token(in, cot);
#pragma unroll
            for (int j = 0; j < W - 1 - t; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) ds[t + j][e] = fmaf(w[j][e], dp[W - 1][e], ds[t + j][e]);
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i) Raw8<T>::of(ds[i]).store(static_cast<T *>(a.ds0) + (b * (W - 1) + i) * a.P + c);
        return;
    }
    int64_t t = (int64_t(blockIdx.x) * rg + at.run) * tr;
    const int64_t stop = at.in ? min(t + tr, a.q.rows) : 0;
    if (a.q.off && t < stop) t = max(t, a.q.at(0));
    while (t < stop) {
        const int64_t b = a.q.find(t);
        if (b < 0) break;
        const int64_t begin = a.q.begin(b), end = a.q.end(b), from = t, last = min(end, stop), until = last + W - 1;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            entry<T, W>(a, b, begin, t - begin + j, c).get(x[j + 1]);
#pragma unroll
            for (int e = 0; e < 8; ++e) dp[j + 1][e] = 0.f;
        }
        Raw8<T> nx[CU], ng[CU];
        auto fetch = [&](int64_t t0) {
#pragma unroll
            for (int u = 0; u < CU; ++u)
                if (t0 + u < min(end, until)) {
                    nx[u].load(row<T>(a.x, t0 + u, a.ldx, c));
                    ng[u].load(row<T>(a.go, t0 + u, a.ldy, c));
                }
        };
        fetch(t);
        for (; t < until; t += CU) {
            Raw8<T> px[CU], pg[CU];
#pragma unroll
            for (int u = 0; u < CU; ++u) {
                px[u] = nx[u];
                pg[u] = ng[u];
            }
            fetch(t + CU);
#pragma unroll
            for (int u = 0; u < CU; ++u) {
                const int64_t tt = t + u, s = tt - (W - 1);
                if (tt >= until) break;
                shift();
                if (tt < end) {
                    token(px[u], pg[u]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) dp[W - 1][e] = 0.f;
                }
                if (tt < last) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        db[e] += dp[W - 1][e];
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][e] = fmaf(dp[W - 1][e], x[j][e], dw[j][e]);
                    }
                }
                if (s >= from) {
                    float d[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) d[e] = 0.f;
                    if (a.ds1 && s >= end - (W - 1)) {
                        Raw8<T> r;
                        r.load(row<T>(a.ds1, b * (W - 1) + (s - end + W - 1), a.P, c));
                        r.get(d);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
#pragma unroll
                        for (int j = 0; j < W; ++j) d[e] = fmaf(w[W - 1 - j][e], dp[j][e], d[e]);
                    Raw8<T>::of(d).store(static_cast<T *>(a.dx) + s * a.ldx + c);
                }
            }
        }
        t = last;
    }
    // the block's sums over its runs, in their order
    const int width = vg * 8, col = int(threadIdx.x) % vg * 8;
    for (int k = 0; k <= W; ++k) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v = db[e];
#pragma unroll
            for (int j = 0; j < W; ++j) v = k == j ? dw[j][e] : v;
            sum[at.run * width + col + e] = v;
        }
        __syncthreads();
        const int p = int(blockIdx.y) * width + int(threadIdx.x);
        if (int(threadIdx.x) < width && p < a.P) {
            float v = 0.f;
            for (int r = 0; r < rg; ++r) v += sum[r * width + threadIdx.x];
            a.part[(int64_t(blockIdx.x) * (W + 1) + k) * a.P + p] = v;
        }
    }
}

// dw [P][W] and dbias from the blocks' sums, in their order
__global__ __launch_bounds__(CT) void k_conv_join(const ConvArgs a, int64_t blocks) {
    const int64_t i = int64_t(blockIdx.x) * CT + threadIdx.x, n = int64_t(a.W + 1) * a.P;
    if (i >= n) return;
    const int k = int(i / a.P), p = int(i - int64_t(k) * a.P);
    float s = 0.f;
#pragma unroll 8
    for (int64_t b = 0; b < blocks; ++b) s += __ldg(a.part + b * n + i);
    if (k < a.W) a.dw[int64_t(p) * a.W + k] = s;
    else if (a.dbias) a.dbias[p] = s;
}

template <class T, int W>
__global__ __launch_bounds__(CT) void k_conv_step(const ConvArgs a, T *state, int64_t n_slots, const int32_t *slots) {
    const int pv = a.P / 8;
    const int64_t i = int64_t(blockIdx.x) * CT + threadIdx.x, b = i / pv;
    if (b >= a.q.B) return;
    const int c = int(i - b * pv) * 8;
    const int64_t slot = slots ? int64_t(__ldg(slots + b)) : b;
    T *y = static_cast<T *>(a.y) + b * a.ldy + c;
    if (slot < 0 || slot >= n_slots) {
        Raw8<T> r;
        r.zero();
        r.store(y);
        return;
    }
    Raw8<T> r[W];
    T *s = state + slot * (W - 1) * a.P + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) r[j] = *reinterpret_cast<const Raw8<T> *>(s + int64_t(j) * a.P);
    r[W - 1].load(row<T>(a.x, b, a.ldx, c));
    float w[W][8], p[8];
    load_taps<W>(a, c, w, p);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float x[8];
        r[j].get(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = fmaf(w[j][e], x[e], p[e]);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) r[j + 1].store(s + int64_t(j) * a.P);
    if (a.act) {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] *= sigmoid_f(p[e]);
    }
    Raw8<T>::of(p).store(y);
}

// vectors side by side in a block, runs of `tr` tokens, blocks of runs
struct ConvGrid {
    int vg, tr;
    int64_t runs;
};
// The longest runs (the fewest tokens read twice) of which there are still `want` threads' worth for
// the loads in flight to cover HBM's latency.
ConvGrid conv_grid(const ConvArgs &a, int longest, int shortest, int64_t want) {
    const int pv = a.P / 8;
    ConvGrid g{1, longest, 0};
    while (g.vg < pv && g.vg < 32) g.vg *= 2;
    while (g.tr > shortest && seq_div(a.q.rows, g.tr) * pv < want) g.tr /= 2;
    g.runs = seq_div(a.q.rows, int64_t(g.tr) * (CT / g.vg));
    return g;
}
ConvGrid fwd_grid(const ConvArgs &a) { return conv_grid(a, 32, 4, 152 * 1024); }
ConvGrid bwd_grid(const ConvArgs &a) { return conv_grid(a, 64, 8, 152 * 384); }

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
    const dim3 grid(unsigned(blocks), unsigned(seq_div(a.P / 8, g.vg)));
    ProfScope p(K_CONV_FWD, st);
    pick(a, bf16, [&](auto t, auto w) { k_conv_fwd<decltype(t), decltype(w)::value><<<grid, CT, 0, st>>>(a, g.vg, g.tr, g.runs); });
    return cudaGetLastError();
}

cudaError_t launch_conv_bwd(const ConvArgs &a, bool bf16, cudaStream_t st) {
    const ConvGrid g = bwd_grid(a);
    const int64_t blocks = g.runs + (a.ds0 ? seq_div(a.q.B, CT / g.vg) : 0);
    if (blocks) {
        const dim3 grid(unsigned(blocks), unsigned(seq_div(a.P / 8, g.vg)));
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
    const unsigned blocks = unsigned(seq_div(a.q.B * (a.P / 8), CT));
    ProfScope p(K_CONV_STEP, st);
    pick(a, bf16, [&](auto t, auto w) {
        typedef decltype(t) T;
        k_conv_step<T, decltype(w)::value><<<blocks, CT, 0, st>>>(a, static_cast<T *>(state), n_slots, slots);
    });
    return cudaGetLastError();
}

}  // namespace adj
