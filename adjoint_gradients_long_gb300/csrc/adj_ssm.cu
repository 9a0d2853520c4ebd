// adj_ssm.cu -- the selective scan with states in and out: prompts, gradients and single tokens.
// include/adj.h defines it.
//
//     h_t = a_t h_{t-1} + u_t B_t,  a_t = exp(d_t A),  u_t = d_t x_t,  v_t = sum_n C_t h_t + D x_t
// and with g_t the cotangent of v_t, m_t that of h_t and e_t = a_t m_t (what reaches h_{t-1}):
//     m_t = g_t C_t + e_{t+1}
//     dB_t = sum_p u m_t      dC_t = sum_p g h_t        dA = sum_t d e_t h_{t-1}
//     dx_t = d sum_n m_t B + D g                        dd_t = x sum_n m_t B + sum_n A e_t h_{t-1}
//
// A warp owns a segment of consecutive tokens for CW = 512 / N channels; a thread owns four
// channels and four states of each, sixteen states in registers.  Lane = quad of states +
// (N / 4) quad of channels.  Pairs of channels go through the packed fp32 instructions; the exponential
// of every state and token, one a lane, is what the pipes have most of.  The inputs of a tile of TT
// tokens are staged in the warp's own part of shared memory, converted to fp32 once (B and C twice
// over, as pairs); sums over states or channels leave through shared memory too, one 16-byte store
// a thread and token, and are added up by whole tiles: a butterfly of shuffles costs three times that.
//
// The tokens are cut into segments, as many as fill the machine.  k_ssm_state walks every segment from
// a state of zero; k_ssm_carry goes over the segments in order and leaves the state that enters each;
// k_ssm_out or k_ssm_grad walk the segments again from there.  One segment needs the last alone.
// The backward pass keeps the state at the start of every tile: the one that k_ssm_state makes from
// zero, plus what enters the segment times exp(A sum d), so no third walk is needed; inside a
// tile the states are formed forwards, kept for four tokens at a time, and used backwards.
//
// Sequences may begin and end anywhere: a tile has a mask of the tokens that begin one (there the state
// is loaded) and of those that end one (there it is stored).  Tokens of no sequence are staged as
// d = u = g = 0, which changes no state and adds to no sum.
#include <algorithm>

#include "adj_lin.cuh"
#include "adj_profile.cuh"
#include "adj_seq.cuh"

namespace adj {
namespace {

constexpr int WPB = 4;                  // warps of a block, side by side in channels
constexpr int G = 4;                    // tokens whose states the backward pass keeps in registers

template <int N>
struct Tile {
    static constexpr int NQ = N / 4, CQ = 32 / NQ, CW = 4 * CQ;
    static constexpr int TT = N == 8 ? 8 : 16;
    static constexpr int QPL = TT * CQ / 32;                        // a lane's quads of channels in a tile
    static constexpr int MAPS = TT * N / 8, MPL = (MAPS + 31) / 32; // vectors of eight of B (or C); a lane's
    static constexpr int X = TT * CW;                               // floats of a tile of channels
    static constexpr int S = TT * N * 2;                            // floats of a tile of B or C, doubled
};
inline int tile_tokens(int N) { return N == 8 ? 8 : 16; }
inline int warp_channels(int N) { return 512 / N; }

// four states of four channels: [state][pair of channels]
struct Quad {
    pair_t v[4][2];
    __device__ __forceinline__ void fill(float x) {
#pragma unroll
        for (int n = 0; n < 4; ++n) v[n][0] = v[n][1] = pk(x, x);
    }
    // channel c, state n of an array [P][N] from `p` on (in: these channels exist)
    template <int N>
    __device__ __forceinline__ void load(const float *p, bool in) {
        float4 r[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) r[c] = in ? *reinterpret_cast<const float4 *>(p + c * N) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            v[0][k] = pk(r[2 * k].x, r[2 * k + 1].x);
            v[1][k] = pk(r[2 * k].y, r[2 * k + 1].y);
            v[2][k] = pk(r[2 * k].z, r[2 * k + 1].z);
            v[3][k] = pk(r[2 * k].w, r[2 * k + 1].w);
        }
    }
    template <int N>
    __device__ __forceinline__ void store(float *p, bool in) const {
        if (!in) return;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float4 x, y;
            upk(v[0][k], x.x, y.x);
            upk(v[1][k], x.y, y.y);
            upk(v[2][k], x.z, y.z);
            upk(v[3][k], x.w, y.w);
            *reinterpret_cast<float4 *>(p + 2 * k * N) = x;
            *reinterpret_cast<float4 *>(p + (2 * k + 1) * N) = y;
        }
    }
};

__device__ __forceinline__ ulonglong2 lds2(const float *p) { return *reinterpret_cast<const ulonglong2 *>(p); }

// A warp's place: its channels, segment and lanes
template <int N>
struct Lane {
    typedef Tile<N> K;
    int lane, nq, cq, warp, c0;         // c0: the warp's first channel
    int64_t seg, col;                   // segment, block of channels
    int64_t t0, t1, lo, hi;             // the segment's tokens; those that belong to sequences
    bool in;                            // this thread's four channels exist
    __device__ Lane(const SsmArgs &a, int64_t block, int64_t cols) {
        lane = threadIdx.x & 31;
        warp = threadIdx.x >> 5;
        nq = lane % K::NQ;
        cq = lane / K::NQ;
        seg = block / cols;
        col = block - seg * cols;
        c0 = int(col * WPB + warp) * K::CW;
        in = c0 + cq * 4 < a.P;
        t0 = seg * a.seglen;
        t1 = min(t0 + a.seglen, a.q.rows);
        lo = t0;
        hi = t1;
        if (a.q.off) {
            lo = max(t0, a.q.at(0));
            hi = min(t1, a.q.at(a.q.B));
        }
    }
    __device__ __forceinline__ int64_t state(const SsmArgs &a) const { return int64_t(c0 + cq * 4) * N + nq * 4; }
    __device__ __forceinline__ const float *of(const SsmArgs &a, const float *base, int64_t i) const {
        return base + i * a.P * N + state(a);
    }
    __device__ __forceinline__ float *of(const SsmArgs &a, float *base, int64_t i) const { return base + i * a.P * N + state(a); }
};

// The sequences of a tile's tokens, bit i (lane i) for token i
struct Marks {
    int64_t b, begin, end;              // a sequence met before: most tiles lie inside it
    uint32_t first, last;
    int64_t seq;                        // of this lane's token
    __device__ Marks() : b(-1), begin(0), end(0) {}
    // forwards: the sequence of the last token is remembered, else that of the first
    template <int TT>
    __device__ void at(const Seqs &q, int64_t t, int64_t lo, int64_t hi, bool forwards) {
        if (b >= 0 && begin <= t && t + TT <= end) {
            first = begin == t ? 1u : 0u;
            last = end == t + TT ? 1u << (TT - 1) : 0u;
            seq = b;
            return;
        }
        const int lane = threadIdx.x & 31;
        const int64_t x = t + lane;
        int64_t s = lane < TT && x >= lo && x < hi ? q.find(x) : -1, s0 = 0, s1 = 0;
        if (s >= 0) {
            s0 = q.begin(s);
            s1 = q.end(s);
        }
        first = __ballot_sync(~0u, s >= 0 && s0 == x);
        last = __ballot_sync(~0u, s >= 0 && s1 == x + 1);
        const uint32_t any = __ballot_sync(~0u, s >= 0);
        seq = s >= 0 ? s : 0;
        if (any) {
            const int l = forwards ? 31 - __clz(any) : __ffs(any) - 1;
            b = __shfl_sync(~0u, s, l);
            begin = __shfl_sync(~0u, s0, l);
            end = __shfl_sync(~0u, s1, l);
        }
    }
    __device__ __forceinline__ int64_t of(int i) const { return __shfl_sync(~0u, seq, i); }
};

// What a lane stages and finishes: quad j is token row + NQ j of the tile, always the same channels
template <class T, int N>
struct Mine {
    typedef Tile<N> K;
    int row, cl, c;                     // cl: channel inside the warp's, c: in the array
    bool in;
    float4 bias, D;
    __device__ Mine(const SsmArgs &a, const Lane<N> &l) {
        row = l.lane / K::CQ;
        cl = l.lane % K::CQ * 4;
        c = l.c0 + cl;
        in = c < a.P;
        bias = a.bias && in ? __ldg(reinterpret_cast<const float4 *>(a.bias + c)) : f4(0.f);
        D = a.D && in ? __ldg(reinterpret_cast<const float4 *>(a.D + c)) : f4(0.f);
    }
    __device__ __forceinline__ int tok(int j) const { return row + K::NQ * j; }
    __device__ __forceinline__ bool ok(const Lane<N> &l, int64_t t, int j) const {
        const int64_t x = t + tok(j);
        return in && x >= l.lo && x < l.hi;
    }
    __device__ __forceinline__ void load(Raw4<T> (&r)[K::QPL], const void *p, int64_t ld, const Lane<N> &l, int64_t t) const {
#pragma unroll
        for (int j = 0; j < K::QPL; ++j) {
            if (ok(l, t, j)) r[j].load(static_cast<const T *>(p) + (t + tok(j)) * ld + c);
            else r[j].zero();
        }
    }
};

__device__ __forceinline__ float4 softplus4(float4 v) {
    return make_float4(softplus_f(v.x), softplus_f(v.y), softplus_f(v.z), softplus_f(v.w));
}
__device__ __forceinline__ void put4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ float4 get4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

// steps and inputs of a tile: d and u = d x (zeros where there is no token)
template <class T, int N>
__device__ __forceinline__ void stage_steps(const Lane<N> &l, const Mine<T, N> &v, int64_t t, const Raw4<T> (&rx)[Tile<N>::QPL],
                                            const Raw4<T> (&rdt)[Tile<N>::QPL], float *ds, float *us) {
    typedef Tile<N> K;
#pragma unroll
    for (int j = 0; j < K::QPL; ++j) {
        const float4 d = v.ok(l, t, j) ? softplus4(rdt[j].get() + v.bias) : f4(0.f);
        put4(ds + v.tok(j) * K::CW + v.cl, d);
        put4(us + v.tok(j) * K::CW + v.cl, d * rx[j].get());
    }
}

// the cotangent g of v: go, times z sigmoid(z) with a gate
template <class T, int N>
__device__ __forceinline__ void stage_cotangent(const SsmArgs &a, const Mine<T, N> &v, const Raw4<T> (&rg)[Tile<N>::QPL],
                                                const Raw4<T> (&rz)[Tile<N>::QPL], float *gs) {
    typedef Tile<N> K;
#pragma unroll
    for (int j = 0; j < K::QPL; ++j) {
        float4 g = rg[j].get();
        if (a.z) {
            const float4 z = rz[j].get();
            g = g * (z * sigmoid4(z));
        }
        put4(gs + v.tok(j) * K::CW + v.cl, g);
    }
}

// B or C of a tile: fetched, and staged with each value twice
template <class T, int N>
struct Maps {
    typedef Tile<N> K;
    Raw8<T> r[K::MPL];
    __device__ __forceinline__ void load(const void *p, int64_t ld, const Lane<N> &l, int64_t t) {
#pragma unroll
        for (int j = 0; j < K::MPL; ++j) {
            const int i = l.lane + 32 * j, tok = i / (N / 8), n = i % (N / 8) * 8;
            if (tok < K::TT && t + tok >= l.lo && t + tok < l.hi) r[j].load(static_cast<const T *>(p) + (t + tok) * ld + n);
            else r[j].zero();
        }
    }
    __device__ __forceinline__ void stage(const Lane<N> &l, float *s) const {
#pragma unroll
        for (int j = 0; j < K::MPL; ++j) {
            const int i = l.lane + 32 * j;
            float x[8];
            r[j].get(x);
            if (i < K::MAPS)
#pragma unroll
                for (int e = 0; e < 8; e += 2) put4(s + (i * 8 + e) * 2, make_float4(x[e], x[e], x[e + 1], x[e + 1]));
        }
    }
};

template <int N>
__device__ __forceinline__ Quad decays(const SsmArgs &a, const Lane<N> &l) {
    Quad A;
    A.load<N>(a.A + l.state(a), l.in);
    const pair_t e = pk(SEQ_LOG2E, SEQ_LOG2E);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) A.v[n][k] = mul2(A.v[n][k], e);
    return A;
}

// The exponential unit's results lie low by 2e-8 on average where the exponent is near zero (measured over
// 0 to -1; 0.3 to 0.8 units of the last place at worst either way).  States that last for a
// thousand tokens would show it, so exponents are raised by that much in the multiply-add that forms them.
constexpr float EXP_UP = 2.5e-8f;

// what a thread reads of a token: its channels' steps and inputs, its states' B (or C)
template <int N>
struct Token {
    pair_t d[2], u[2], B[4];
    __device__ __forceinline__ void load(const float *ds, const float *us, const float *Bs, const Lane<N> &l, int i) {
        const ulonglong2 x = lds2(ds + i * Tile<N>::CW + l.cq * 4), y = lds2(us + i * Tile<N>::CW + l.cq * 4);
        d[0] = x.x; d[1] = x.y;
        u[0] = y.x; u[1] = y.y;
        maps(B, Bs, l, i);
    }
    __device__ __forceinline__ static void maps(pair_t (&b)[4], const float *s, const Lane<N> &l, int i) {
        const ulonglong2 x = lds2(s + (i * N + l.nq * 4) * 2), y = lds2(s + (i * N + l.nq * 4) * 2 + 4);
        b[0] = x.x; b[1] = x.y; b[2] = y.x; b[3] = y.y;
    }
};

// h = exp(d A) h + u B for one token
template <bool KEEP, int N>
__device__ __forceinline__ void advance(const Quad &A, Quad &h, Quad *keep, const Token<N> &k) {
    const pair_t up = pk(EXP_UP, EXP_UP);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const pair_t e = exp2_2(fma2(k.d[c], A.v[n][c], up));
            if (KEEP) keep->v[n][c] = e;
            h.v[n][c] = fma2(e, h.v[n][c], mul2(k.u[c], k.B[n]));
        }
}

// ---------------------------------------------------------------- segments from a state of zero
template <class T, int N, bool BWD>
__global__ __launch_bounds__(32 * WPB, 3) void k_ssm_state(const SsmArgs a, int64_t cols) {
    typedef Tile<N> K;
    extern __shared__ __align__(16) float sm[];
    const Lane<N> l(a, blockIdx.x, cols);
    const Mine<T, N> v(a, l);
    float *ds = sm + l.warp * ((BWD ? 3 : 2) * K::X + (BWD ? 2 : 1) * K::S), *us = ds + K::X, *Bs = us + K::X;
    float *Cs = Bs + K::S, *gs = Cs + K::S;                         // BWD
    const Quad A = decays<N>(a, l);
    Quad h, P, m;
    h.fill(0.f);
    P.fill(1.f);
    m.fill(0.f);
    pair_t sum[2] = {pk(0.f, 0.f), pk(0.f, 0.f)};
    bool fresh = false;                                             // a sequence has begun in this segment
    Marks mk;
    Raw4<T> rx[K::QPL], rdt[K::QPL];
    Maps<T, N> rB;
    v.load(rx, a.x, a.ldx, l, l.t0);
    v.load(rdt, a.dt, a.lddt, l, l.t0);
    rB.load(a.Bm, a.ldB, l, l.t0);
    auto steps = [&](float *p) {                                    // [P] of the sums of steps
        if (l.nq != 0 || !l.in) return;
        float4 s;
        upk(sum[0], s.x, s.y);
        upk(sum[1], s.z, s.w);
        put4(p + l.c0 + l.cq * 4, fresh ? f4(-1.f) : s);
    };
    for (int64_t t = l.t0; t < l.t1; t += K::TT) {
        if (BWD) {
            const int64_t tile = t / K::TT;
            h.store<N>(l.of(a, a.tile, tile), l.in);
            steps(a.tstep + tile * a.P);
        }
        mk.at<K::TT>(a.q, t, l.lo, l.hi, true);
        __syncwarp();
        stage_steps<T, N>(l, v, t, rx, rdt, ds, us);
        rB.stage(l, Bs);
        if (BWD) {
            Raw4<T> rg[K::QPL], rz[K::QPL];
            Maps<T, N> rC;
            v.load(rg, a.go, a.ldy, l, t);
            if (a.z) v.load(rz, a.z, a.ldz, l, t);
            rC.load(a.Cm, a.ldC, l, t);
            stage_cotangent<T, N>(a, v, rg, rz, gs);
            rC.stage(l, Cs);
        }
        __syncwarp();
        v.load(rx, a.x, a.ldx, l, t + K::TT);
        v.load(rdt, a.dt, a.lddt, l, t + K::TT);
        rB.load(a.Bm, a.ldB, l, t + K::TT);
        auto walk = [&](auto events, int i0) {
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const int i = i0 + j;
                Token<N> k;
                k.load(ds, us, Bs, l, i);
                if (events && (mk.first >> i & 1u)) {
                    const int64_t b = mk.of(i);
                    if (a.s0) h.load<N>(l.of(a, a.s0, b), l.in);
                    else h.fill(0.f);
                    fresh = true;
                }
                sum[0] = add2(sum[0], k.d[0]);
                sum[1] = add2(sum[1], k.d[1]);
                Quad e;
                advance<BWD>(A, h, &e, k);
                if (BWD && !(events && fresh)) {
                    const ulonglong2 g = lds2(gs + i * K::CW + l.cq * 4);
                    const pair_t gg[2] = {g.x, g.y};
                    pair_t C[4];
                    Token<N>::maps(C, Cs, l, i);
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            P.v[n][c] = mul2(P.v[n][c], e.v[n][c]);
                            m.v[n][c] = fma2(P.v[n][c], mul2(gg[c], C[n]), m.v[n][c]);
                        }
                    if (events && a.ds1 && (mk.last >> i & 1u)) {
                        Quad s;
                        s.load<N>(l.of(a, a.ds1, mk.of(i)), l.in);
#pragma unroll
                        for (int n = 0; n < 4; ++n)
#pragma unroll
                            for (int c = 0; c < 2; ++c) m.v[n][c] = fma2(P.v[n][c], s.v[n][c], m.v[n][c]);
                    }
                }
            }
        };
#pragma unroll 1
        for (int i = 0; i < K::TT; i += G) {
            if (((mk.first | mk.last) >> i & ((1u << G) - 1)) || (BWD && fresh)) walk(std::true_type(), i);
            else walk(std::false_type(), i);
        }
    }
    h.store<N>(l.of(a, a.seg, l.seg), l.in);
    steps(a.step + l.seg * a.P);
    if (BWD) m.store<N>(l.of(a, a.adj, l.seg), l.in);
}

// Over the segments in order: seg becomes the state that enters each; blockIdx.y 1: adj, from the right.
__global__ __launch_bounds__(128) void k_ssm_carry(const SsmArgs a) {
    const int64_t i = int64_t(blockIdx.x) * 128 + threadIdx.x, n = int64_t(a.P) * a.N / 4;
    if (i >= n) return;
    const bool right = blockIdx.y != 0;
    const int p = int(i / (a.N / 4));
    const float4 A = f4(SEQ_LOG2E) * __ldg(reinterpret_cast<const float4 *>(a.A) + i);
    float4 *x = reinterpret_cast<float4 *>(right ? a.adj : a.seg) + i, cur = f4(0.f);
    constexpr int U = 8;
    for (int64_t s0 = 0; s0 < a.nseg; s0 += U) {
        float4 v[U];
        float d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t s = right ? a.nseg - 1 - (s0 + u) : s0 + u;
            if (s0 + u < a.nseg) {
                v[u] = x[s * n];
                d[u] = a.step[s * a.P + p];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t s = right ? a.nseg - 1 - (s0 + u) : s0 + u;
            if (s0 + u < a.nseg) {
                x[s * n] = cur;
                cur = d[u] < 0.f ? v[u]
                                 : fma4(make_float4(fast_exp2(A.x * d[u]), fast_exp2(A.y * d[u]), fast_exp2(A.z * d[u]),
                                                    fast_exp2(A.w * d[u])), cur, v[u]);
            }
        }
    }
}

// The states of sequences without tokens pass through (out: s1 or ds0, in: s0 or ds1); block `e` of `of`.
__device__ void pass_through(const SsmArgs &a, float *out, const float *in, int64_t e, int64_t of) {
    const int64_t n = int64_t(a.P) * a.N / 4;
    for (int64_t b = e; b < a.q.B; b += of) {
        if (a.q.begin(b) < a.q.end(b)) continue;
        for (int64_t i = threadIdx.x; i < n; i += blockDim.x)
            reinterpret_cast<float4 *>(out)[b * n + i] = in ? reinterpret_cast<const float4 *>(in)[b * n + i] : f4(0.f);
    }
}

// ---------------------------------------------------------------- outputs
template <class T, int N>
__global__ __launch_bounds__(32 * WPB, 3) void k_ssm_out(const SsmArgs a, int64_t cols) {
    typedef Tile<N> K;
    extern __shared__ __align__(16) float sm[];
    const int64_t work = a.nseg * cols;
    if (int64_t(blockIdx.x) >= work) {
        pass_through(a, a.s1, a.s0, blockIdx.x - work, gridDim.x - work);
        return;
    }
    const Lane<N> l(a, blockIdx.x, cols);
    const Mine<T, N> v(a, l);
    float *ds = sm + l.warp * (2 * K::X + 2 * K::S + K::TT * 128), *us = ds + K::X, *Bs = us + K::X, *Cs = Bs + K::S;
    float *ys = Cs + K::S;                                          // [TT][NQ][CW]: sums over a quad of states
    const Quad A = decays<N>(a, l);
    Quad h;
    h.fill(0.f);
    if (a.nseg > 1) h.load<N>(l.of(a, a.seg, l.seg), l.in);
    Marks mk;
    Raw4<T> rx[K::QPL], rdt[K::QPL], rz[K::QPL], cx[K::QPL];
    Maps<T, N> rB, rC;
    auto fetch = [&](int64_t t) {
        v.load(rx, a.x, a.ldx, l, t);
        v.load(rdt, a.dt, a.lddt, l, t);
        rB.load(a.Bm, a.ldB, l, t);
        rC.load(a.Cm, a.ldC, l, t);
    };
    fetch(l.t0);
    for (int64_t t = l.t0; t < l.t1; t += K::TT) {
        mk.at<K::TT>(a.q, t, l.lo, l.hi, true);
        __syncwarp();
        stage_steps<T, N>(l, v, t, rx, rdt, ds, us);
        rB.stage(l, Bs);
        rC.stage(l, Cs);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < K::QPL; ++j) cx[j] = rx[j];
        if (a.z) v.load(rz, a.z, a.ldz, l, t);
        fetch(t + K::TT);
        // the sums of a group stay in registers until its end: a store to shared memory would hold up
        // the next token's loads
        auto walk = [&](auto events, int i0) {
            ulonglong2 y[G];
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const int i = i0 + j;
                Token<N> k;
                pair_t C[4];
                k.load(ds, us, Bs, l, i);
                Token<N>::maps(C, Cs, l, i);
                if (events && (mk.first >> i & 1u)) {
                    const int64_t b = mk.of(i);
                    if (a.s0) h.load<N>(l.of(a, a.s0, b), l.in);
                    else h.fill(0.f);
                }
                advance<false>(A, h, nullptr, k);
                y[j].x = mul2(C[0], h.v[0][0]);
                y[j].y = mul2(C[0], h.v[0][1]);
#pragma unroll
                for (int n = 1; n < 4; ++n) {
                    y[j].x = fma2(C[n], h.v[n][0], y[j].x);
                    y[j].y = fma2(C[n], h.v[n][1], y[j].y);
                }
                if (events && a.s1 && (mk.last >> i & 1u)) {
                    const int64_t b = mk.of(i);
                    h.store<N>(l.of(a, a.s1, b), l.in);
                }
            }
#pragma unroll
            for (int j = 0; j < G; ++j)
                *reinterpret_cast<ulonglong2 *>(ys + ((i0 + j) * K::NQ + l.nq) * K::CW + l.cq * 4) = y[j];
        };
#pragma unroll 1
        for (int i = 0; i < K::TT; i += G) {
            if ((mk.first | mk.last) >> i & ((1u << G) - 1)) walk(std::true_type(), i);
            else walk(std::false_type(), i);
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < K::QPL; ++j) {
            if (!v.ok(l, t, j)) continue;
            const float *p = ys + v.tok(j) * 128 + v.cl;
            float4 y = get4(p);
#pragma unroll
            for (int q = 1; q < K::NQ; ++q) y = y + get4(p + q * K::CW);
            y = fma4(v.D, cx[j].get(), y);
            if (a.z) {
                const float4 z = rz[j].get();
                y = y * (z * sigmoid4(z));
            }
            st4(static_cast<T *>(a.y) + (t + v.tok(j)) * a.ldy + v.c, y);
        }
    }
}

// ---------------------------------------------------------------- gradients
template <int N>
struct GradSm {                         // floats of a warp's part
    typedef Tile<N> K;
    static constexpr int CK = K::TT / G * 512;                      // states at every G-th token, [.][4][32] x 4
    static constexpr int BC = G * 2 * 128, CH = G * 3 * 128;        // a group's sums: over channels, over states
    static constexpr int SUM = K::TT * 2 * N;                       // dB and dC of a tile over the warp's channels
    static constexpr int ALL = 3 * K::X + 2 * K::S + CK + BC + CH + SUM;
};

template <class T, int N>
__global__ __launch_bounds__(32 * WPB) void k_ssm_grad(const SsmArgs a, int64_t cols) {
    typedef Tile<N> K;
    typedef GradSm<N> M;
    extern __shared__ __align__(16) float sm[];
    const int64_t work = a.nseg * cols;
    if (int64_t(blockIdx.x) >= work) {
        pass_through(a, a.ds0, a.ds1, blockIdx.x - work, gridDim.x - work);
        return;
    }
    const Lane<N> l(a, blockIdx.x, cols);
    const Mine<T, N> v(a, l);
    float *ds = sm + l.warp * M::ALL, *us = ds + K::X, *gs = us + K::X, *Bs = gs + K::X, *Cs = Bs + K::S;
    float *ck = Cs + K::S, *bc = ck + M::CK, *ch = bc + M::BC, *ws = ch + M::CH;
    const Quad A = decays<N>(a, l);
    Quad e, dA;                                                     // e: what reaches the state before
    e.load<N>(l.of(a, a.adj, l.seg), l.in);
    dA.fill(0.f);
    float4 dD = f4(0.f), db = f4(0.f);
    Marks mk;
    const int tiles = int((l.t1 - l.t0 + K::TT - 1) / K::TT);
    for (int ti = tiles - 1; ti >= 0; --ti) {
        const int64_t t = l.t0 + int64_t(ti) * K::TT, tile = t / K::TT;
        mk.at<K::TT>(a.q, t, l.lo, l.hi, false);
        // the state before the tile
        Quad h;
        {
            Quad in;
            float4 s = make_float4(-1.f, -1.f, -1.f, -1.f);
            h.load<N>(l.of(a, a.tile, tile), l.in);
            in.load<N>(l.of(a, a.seg, l.seg), l.in);
            if (l.in) s = *reinterpret_cast<const float4 *>(a.tstep + tile * a.P + l.c0 + l.cq * 4);
            if (s.x >= 0.f) {
                const pair_t d[2] = {pk(s.x, s.y), pk(s.z, s.w)};
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int k = 0; k < 2; ++k) h.v[n][k] = fma2(exp2_2(mul2(d[k], A.v[n][k])), in.v[n][k], h.v[n][k]);
            }
        }
        {
            Raw4<T> rx[K::QPL], rdt[K::QPL], rg[K::QPL], rz[K::QPL];
            Maps<T, N> rB, rC;
            v.load(rx, a.x, a.ldx, l, t);
            v.load(rdt, a.dt, a.lddt, l, t);
            v.load(rg, a.go, a.ldy, l, t);
            if (a.z) v.load(rz, a.z, a.ldz, l, t);
            rB.load(a.Bm, a.ldB, l, t);
            rC.load(a.Cm, a.ldC, l, t);
            __syncwarp();
            stage_steps<T, N>(l, v, t, rx, rdt, ds, us);
            stage_cotangent<T, N>(a, v, rg, rz, gs);
            rB.stage(l, Bs);
            rC.stage(l, Cs);
            __syncwarp();
        }
        auto begin = [&](int i, Quad &x) {                          // the state before a sequence's first token
            const int64_t b = mk.of(i);
            if (a.s0) x.load<N>(l.of(a, a.s0, b), l.in);
            else x.fill(0.f);
        };
        auto keep = [&](int g, const Quad &x) {
#pragma unroll
            for (int n = 0; n < 4; ++n)
                *reinterpret_cast<ulonglong2 *>(ck + ((g * 4 + n) * 32 + l.lane) * 4) = make_ulonglong2(x.v[n][0], x.v[n][1]);
        };
        keep(0, h);
        for (int g = 1; g < K::TT / G; ++g) {
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const int i = (g - 1) * G + j;
                if (mk.first >> i & 1u) begin(i, h);
                Token<N> k;
                k.load(ds, us, Bs, l, i);
                advance<false>(A, h, nullptr, k);
            }
            keep(g, h);
        }
        for (int g = K::TT / G - 1; g >= 0; --g) {
            Quad hp[G], ea[G];                                      // the state before each token, its decay
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const ulonglong2 x = lds2(ck + ((g * 4 + n) * 32 + l.lane) * 4);
                h.v[n][0] = x.x;
                h.v[n][1] = x.y;
            }
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const int i = g * G + j;
                if (mk.first >> i & 1u) begin(i, h);
                hp[j] = h;
                Token<N> k;
                k.load(ds, us, Bs, l, i);
                advance<true>(A, h, &ea[j], k);
            }
#pragma unroll
            for (int j = G - 1; j >= 0; --j) {
                const int i = g * G + j;
                const float *Bi = Bs + (i * N + l.nq * 4) * 2, *Ci = Cs + (i * N + l.nq * 4) * 2;
                const ulonglong2 d2 = lds2(ds + i * K::CW + l.cq * 4), u2 = lds2(us + i * K::CW + l.cq * 4);
                const ulonglong2 g2 = lds2(gs + i * K::CW + l.cq * 4), b0 = lds2(Bi), b1 = lds2(Bi + 4), c0 = lds2(Ci), c1 = lds2(Ci + 4);
                const pair_t d[2] = {d2.x, d2.y}, u[2] = {u2.x, u2.y}, gg[2] = {g2.x, g2.y};
                const pair_t B[4] = {b0.x, b0.y, b1.x, b1.y}, C[4] = {c0.x, c0.y, c1.x, c1.y};
                if (mk.last >> i & 1u) {
                    const int64_t b = mk.of(i);
                    if (a.ds1) e.load<N>(l.of(a, a.ds1, b), l.in);
                    else e.fill(0.f);
                }
                const pair_t zero = pk(0.f, 0.f);
                pair_t vv[2] = {zero, zero}, mb[2] = {zero, zero}, sa[2] = {zero, zero};
                float dB[4], dC[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    pair_t xb = zero, xc = zero;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        // the state after the token; the next one's is another sequence's where that begins
                        const pair_t hn = fma2(ea[j].v[n][k], hp[j].v[n][k], mul2(u[k], B[n]));
                        const pair_t m = fma2(gg[k], C[n], e.v[n][k]);
                        vv[k] = fma2(C[n], hn, vv[k]);
                        xc = fma2(gg[k], hn, xc);
                        xb = fma2(u[k], m, xb);
                        mb[k] = fma2(m, B[n], mb[k]);
                        e.v[n][k] = mul2(ea[j].v[n][k], m);
                        const pair_t w = mul2(e.v[n][k], hp[j].v[n][k]);
                        dA.v[n][k] = fma2(w, d[k], dA.v[n][k]);
                        sa[k] = fma2(w, A.v[n][k], sa[k]);
                    }
                    float x, y;
                    upk(xb, x, y);
                    dB[n] = x + y;
                    upk(xc, x, y);
                    dC[n] = x + y;
                }
                *reinterpret_cast<float4 *>(bc + (j * 2 + 0) * 128 + l.cq * N + l.nq * 4) = make_float4(dB[0], dB[1], dB[2], dB[3]);
                *reinterpret_cast<float4 *>(bc + (j * 2 + 1) * 128 + l.cq * N + l.nq * 4) = make_float4(dC[0], dC[1], dC[2], dC[3]);
                *reinterpret_cast<ulonglong2 *>(ch + (j * 3 + 0) * 128 + l.nq * K::CW + l.cq * 4) = make_ulonglong2(mb[0], mb[1]);
                *reinterpret_cast<ulonglong2 *>(ch + (j * 3 + 1) * 128 + l.nq * K::CW + l.cq * 4) = make_ulonglong2(sa[0], sa[1]);
                *reinterpret_cast<ulonglong2 *>(ch + (j * 3 + 2) * 128 + l.nq * K::CW + l.cq * 4) = make_ulonglong2(vv[0], vv[1]);
                if (mk.first >> i & 1u) {
                    const int64_t b = mk.of(i);
                    if (a.ds0) e.store<N>(l.of(a, a.ds0, b), l.in);
                    e.fill(0.f);
                }
            }
            __syncwarp();
            // the group's sums: over states into ds, us, gs (done with), over channels into ws
            for (int x = l.lane; x < G * 3 * K::CQ; x += 32) {
                const int q = x % K::CQ, r = x / K::CQ, kind = r % 3, j = r / 3;
                const float4 *p = reinterpret_cast<const float4 *>(ch + r * 128 + q * 4);
                float4 s = p[0];
#pragma unroll
                for (int y = 1; y < K::NQ; ++y) s = s + p[y * K::CW / 4];
                float *to = kind == 0 ? ds : kind == 1 ? us : gs;
                *reinterpret_cast<float4 *>(to + (g * G + j) * K::CW + q * 4) = s;
            }
            for (int x = l.lane; x < G * 2 * K::NQ; x += 32) {
                const int q = x % K::NQ, r = x / K::NQ, kind = r % 2, j = r / 2;
                const float4 *p = reinterpret_cast<const float4 *>(bc + r * 128 + q * 4);
                float4 s = p[0];
#pragma unroll
                for (int y = 1; y < K::CQ; ++y) s = s + p[y * N / 4];
                *reinterpret_cast<float4 *>(ws + (g * G + j) * 2 * N + kind * N + q * 4) = s;
            }
            __syncwarp();
        }
        // the tile's gradients of what each channel reads
        {
            Raw4<T> rx[K::QPL], rdt[K::QPL], rz[K::QPL], rg[K::QPL];
            v.load(rx, a.x, a.ldx, l, t);
            v.load(rdt, a.dt, a.lddt, l, t);
            v.load(rg, a.go, a.ldy, l, t);
            if (a.z) v.load(rz, a.z, a.ldz, l, t);
#pragma unroll
            for (int j = 0; j < K::QPL; ++j) {
                if (!v.ok(l, t, j)) continue;
                const int64_t at = t + v.tok(j);
                const int sh = v.tok(j) * K::CW + v.cl;
                const float4 x = rx[j].get(), raw = rdt[j].get() + v.bias, mb = get4(ds + sh);
                float4 g = rg[j].get();
                if (a.z) {
                    // v z s: its derivative for z is v s (1 + z (1 - s))
                    const float4 z = rz[j].get(), s = sigmoid4(z), val = fma4(v.D, x, get4(gs + sh));
                    st4(static_cast<T *>(a.dz) + at * a.ldz + v.c, g * val * s * fma4(z, f4(1.f) - s, f4(1.f)));
                    g = g * (z * s);
                }
                const float4 ddt = fma4(x, mb, f4(SEQ_LN2) * get4(us + sh)) * sigmoid4(raw);
                st4(static_cast<T *>(a.dx) + at * a.ldx + v.c, fma4(softplus4(raw), mb, v.D * g));
                st4(static_cast<T *>(a.ddt) + at * a.lddt + v.c, ddt);
                dD = fma4(g, x, dD);
                db = db + ddt;
            }
        }
        // dB and dC over the block's warps
        __syncthreads();
        for (int x = threadIdx.x; x < K::TT * N / 2; x += 32 * WPB) {
            const int tok = x / (N / 2), q = x % (N / 2) * 4;
            const float *p = sm + (M::ALL - M::SUM) + tok * 2 * N + q;
            float4 s = *reinterpret_cast<const float4 *>(p);
#pragma unroll
            for (int w = 1; w < WPB; ++w) s = s + *reinterpret_cast<const float4 *>(p + w * M::ALL);
            if (t + tok < l.t1) *reinterpret_cast<float4 *>(a.bc + ((l.col * a.q.rows + t + tok) * 2 * N + q)) = s;
        }
        __syncthreads();
    }
    float *par = a.par + l.seg * a.P * (N + 2);
    dA.store<N>(par + l.state(a), l.in);
#pragma unroll
    for (int w = K::CQ; w < 32; w <<= 1) {
        auto join = [&](float4 &x) {
            x = x + make_float4(__shfl_xor_sync(~0u, x.x, w), __shfl_xor_sync(~0u, x.y, w), __shfl_xor_sync(~0u, x.z, w),
                                __shfl_xor_sync(~0u, x.w, w));
        };
        join(dD);
        join(db);
    }
    if (l.lane < K::CQ && v.in) {
        put4(par + int64_t(a.P) * N + v.c, dD);
        put4(par + int64_t(a.P) * (N + 1) + v.c, db);
    }
}

// The partial sums, each in a fixed order: blocks below `maps` take dB and dC (four values a thread),
// those above the parameters (one value a thread).
template <class T>
__global__ __launch_bounds__(256) void k_ssm_join(const SsmArgs a, int64_t cols, int64_t maps) {
    const int N = a.N;
    if (int64_t(blockIdx.x) < maps) {
        const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x, t = i / (N / 2);
        const int q = int(i - t * (N / 2)) * 4;
        if (t >= a.q.rows || (a.q.off && (t < a.q.at(0) || t >= a.q.at(a.q.B)))) return;
        float4 s = f4(0.f);
#pragma unroll 8
        for (int64_t c = 0; c < cols; ++c) s = s + *reinterpret_cast<const float4 *>(a.bc + (c * a.q.rows + t) * 2 * N + q);
        T *to = q < N ? static_cast<T *>(a.dB) + t * a.ldB + q : static_cast<T *>(a.dC) + t * a.ldC + q - N;
        st4(to, s);
        return;
    }
    const int64_t i = (blockIdx.x - maps) * 256 + threadIdx.x, n = int64_t(a.P) * N, all = n + 2 * int64_t(a.P);
    if (i >= all) return;
    float s = 0.f;
#pragma unroll 8
    for (int64_t g = 0; g < a.nseg; ++g) s += __ldg(a.par + g * all + i);
    if (i < n) a.dA[i] = s;
    else if (i < n + a.P) {
        if (a.dD) a.dD[i - n] = s;
    } else if (a.dbias) a.dbias[i - n - a.P] = s;
}

// ---------------------------------------------------------------- single tokens
// A thread takes four states of each of K channels, K the number of quads of states, 4 at most: its K loads of
// the state are in flight together, and the steps of the K channels are formed by one lane each.
// The state is read and written once, bound by HBM.
template <class T, int N>
__global__ __launch_bounds__(256) void k_ssm_step(const SsmArgs a, float *state, int64_t n_slots, const int32_t *slots) {
    constexpr int NQ = N / 4, K = NQ < 4 ? NQ : 4;
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x, per = int64_t(a.P) / K * NQ, b = i / per;
    if (b >= a.q.B) return;                                         // whole groups of NQ lanes
    const int r = int(i - b * per), nq = r % NQ, c0 = r / NQ * K, k0 = nq % K, p = c0 + k0;
    const uint32_t group = (NQ == 32 ? ~0u : (1u << NQ) - 1) << (threadIdx.x & 31 & ~(NQ - 1));
    T *y = static_cast<T *>(a.y) + b * a.ldy + p;
    const int64_t slot = slots ? int64_t(__ldg(slots + b)) : b;
    if (slot < 0 || slot >= n_slots) {                              // the whole group
        if (nq < K) *y = T(0.f);
        return;
    }
    float4 *s = reinterpret_cast<float4 *>(state + (slot * a.P + c0) * N) + nq, h[K];
#pragma unroll
    for (int k = 0; k < K; ++k) h[k] = s[k * NQ];
    const float x = float(static_cast<const T *>(a.x)[b * a.ldx + p]);
    const float raw = float(static_cast<const T *>(a.dt)[b * a.lddt + p]);
    const float z = a.z ? float(static_cast<const T *>(a.z)[b * a.ldz + p]) : 0.f;
    Raw4<T> rB, rC;
    rB.load(static_cast<const T *>(a.Bm) + b * a.ldB + nq * 4);
    rC.load(static_cast<const T *>(a.Cm) + b * a.ldC + nq * 4);
    const float4 B = rB.get(), C = rC.get(), up = f4(EXP_UP);
    const float d0 = softplus_f(raw + (a.bias ? __ldg(a.bias + p) : 0.f)), u0 = d0 * x;
    float v[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const float d = __shfl_sync(group, d0, k, NQ), u = __shfl_sync(group, u0, k, NQ);
        const float4 A = f4(SEQ_LOG2E) * __ldg(reinterpret_cast<const float4 *>(a.A + int64_t(c0 + k) * N) + nq), t = fma4(f4(d), A, up);
        h[k] = fma4(make_float4(fast_exp2(t.x), fast_exp2(t.y), fast_exp2(t.z), fast_exp2(t.w)), h[k], f4(u) * B);
        s[k * NQ] = h[k];
        v[k] = fmaf(C.x, h[k].x, fmaf(C.y, h[k].y, fmaf(C.z, h[k].z, C.w * h[k].w)));
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int w = 1; w < NQ; w <<= 1) v[k] += __shfl_xor_sync(group, v[k], w);
    if (nq >= K) return;
    float out = v[0];
#pragma unroll
    for (int k = 1; k < K; ++k) out = k0 == k ? v[k] : out;
    if (a.D) out = fmaf(__ldg(a.D + p), x, out);
    if (a.z) out *= z * sigmoid_f(z);
    *y = T(out);
}

// ---------------------------------------------------------------- launches
template <class F>
cudaError_t pick(int N, bool bf16, F f) {
    using std::integral_constant;
    auto sizes = [&](auto t) {
        switch (N) {
            case 8: return f(t, integral_constant<int, 8>());
            case 16: return f(t, integral_constant<int, 16>());
            case 32: return f(t, integral_constant<int, 32>());
            default: return f(t, integral_constant<int, 64>());
        }
    };
    return bf16 ? sizes(__nv_bfloat16()) : sizes(0.f);
}

int64_t columns(const SsmArgs &a) { return seq_div(a.P, WPB * warp_channels(a.N)); }
// blocks that look for sequences without tokens: only packed ones may have any, or all of them have none
int64_t lookers(const SsmArgs &a, const float *out) {
    return out && a.q.B && (a.q.off || a.q.rows == 0) ? std::min<int64_t>(a.q.B, 152) : 0;
}

template <auto Kern>
cudaError_t go(KernelId id, int64_t blocks, size_t smem, cudaStream_t st, const SsmArgs &a, int64_t cols) {
    const cudaError_t e = allow_smem<Kern>();
    if (e != cudaSuccess) return e;
    ProfScope p(id, st);
    Kern<<<unsigned(blocks), 32 * WPB, smem, st>>>(a, cols);
    return cudaGetLastError();
}

cudaError_t carry(const SsmArgs &a, int dirs, cudaStream_t st) {
    ProfScope p(K_SSM_CARRY, st);
    k_ssm_carry<<<dim3(unsigned(seq_div(int64_t(a.P) * a.N / 4, 128)), dirs), 128, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t ssm_plan(SsmArgs &a, bool bwd, void *base) {
    const int64_t tt = tile_tokens(a.N), cols = columns(a), tiles = seq_div(a.q.rows, tt);
    // one turn of the machine: 3 blocks an SM forwards, 2 backwards; short prompts stay in one segment, as
    // a walk of 256 tokens costs less than two more launches
    const int64_t want = std::max<int64_t>(1, 152 * (bwd ? 2 : 3) / cols);
    const int64_t least = bwd ? 2 : a.q.rows <= 256 ? 16 : 4;          // tiles of a segment
    const int64_t per = std::max(least, seq_div(tiles, want));
    a.seglen = per * tt;
    a.nseg = seq_div(a.q.rows, a.seglen);
    char *p = static_cast<char *>(base);
    size_t used = 0;
    auto take = [&](float *&to, int64_t n) {
        to = base ? reinterpret_cast<float *>(p + used) : nullptr;
        used += (size_t(n) * sizeof(float) + 255) & ~size_t(255);
    };
    const int64_t PN = int64_t(a.P) * a.N;
    if (bwd || a.nseg > 1) {
        take(a.seg, a.nseg * PN);
        take(a.step, a.nseg * a.P);
    }
    if (bwd) {
        take(a.adj, a.nseg * PN);
        take(a.tile, tiles * PN);
        take(a.tstep, tiles * a.P);
        take(a.bc, cols * a.q.rows * 2 * a.N);
        take(a.par, a.nseg * (PN + 2 * int64_t(a.P)));
    }
    return used;
}

cudaError_t launch_ssm_fwd(const SsmArgs &a, bool bf16, cudaStream_t st) {
    const int64_t cols = columns(a), look = lookers(a, a.s1);
    return pick(a.N, bf16, [&](auto t, auto n) {
        typedef decltype(t) T;
        constexpr int N = decltype(n)::value;
        typedef Tile<N> K;
        if (a.nseg > 1) {
            LIN_CUDA((go<k_ssm_state<T, N, false>>(K_SSM_STATE, a.nseg * cols, WPB * (2 * K::X + K::S) * 4, st, a, cols)));
            LIN_CUDA(carry(a, 1, st));
        }
        if (a.nseg * cols + look == 0) return cudaSuccess;
        return go<k_ssm_out<T, N>>(K_SSM_OUT, a.nseg * cols + look, WPB * (2 * K::X + 2 * K::S + K::TT * 128) * 4, st, a, cols);
    });
}

cudaError_t launch_ssm_bwd(const SsmArgs &a, bool bf16, cudaStream_t st) {
    const int64_t cols = columns(a), look = lookers(a, a.ds0);
    return pick(a.N, bf16, [&](auto t, auto n) {
        typedef decltype(t) T;
        constexpr int N = decltype(n)::value;
        typedef Tile<N> K;
        if (a.nseg) {
            LIN_CUDA((go<k_ssm_state<T, N, true>>(K_SSM_STATE, a.nseg * cols, WPB * (3 * K::X + 2 * K::S) * 4, st, a, cols)));
            LIN_CUDA(carry(a, 2, st));
        }
        if (a.nseg * cols + look)
            LIN_CUDA((go<k_ssm_grad<T, N>>(K_SSM_GRAD, a.nseg * cols + look, WPB * GradSm<N>::ALL * 4, st, a, cols)));
        const int64_t maps = seq_div(a.q.rows * (N / 2), 256), rest = seq_div(int64_t(a.P) * (N + 2), 256);
        ProfScope p(K_SSM_JOIN, st);
        k_ssm_join<T><<<unsigned(maps + rest), 256, 0, st>>>(a, cols, maps);
        return cudaGetLastError();
    });
}

cudaError_t launch_ssm_step(const SsmArgs &a, bool bf16, float *state, int64_t n_slots, const int32_t *slots,
                            cudaStream_t st) {
    return pick(a.N, bf16, [&](auto t, auto n) {
        typedef decltype(t) T;
        constexpr int N = decltype(n)::value;
        ProfScope p(K_SSM_STEP, st);
        k_ssm_step<T, N><<<unsigned(seq_div(a.q.B * (a.P / std::min(4, N / 4)) * (N / 4), 256)), 256, 0, st>>>(a, state, n_slots, slots);
        return cudaGetLastError();
    });
}

}  // namespace adj
