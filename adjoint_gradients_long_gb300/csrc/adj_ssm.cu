// adj_ssm.cu -- the selective scan with states in and out: prompts, gradients and single tokens.
// include/adj.h defines it.
//
//     h_t = a_t h_{t-1} + u_t B_t,  a_t = exp(d_t A),  u_t = d_t x_t,  v_t = sum_n C_t h_t + D x_t
// and with g_t the cotangent of v_t, m_t that of h_t and e_t = a_t m_t (what reaches h_{t-1}):
//     m_t = g_t C_t + e_{t+1}
//     dB_t = sum_p u m_t      dC_t = sum_p g h_t        dA = sum_t d e_t h_{t-1}
//     dx_t = d sum_n m_t B + D g                        dd_t = x sum_n m_t B + sum_n A e_t h_{t-1}
//
// A warp owns a segment of consecutive tokens for CW channels; a thread owns 2 NP channels and four states
// of each in registers (NP 2; 1 for short prompts).  Lane = quad of states + (N / 4) group of channels.
// Pairs of channels go through the packed fp32 instructions.  The inputs of a tile of TT tokens are
// staged in the warp's own part of shared memory, converted to fp32 once.  A 16-byte load of it takes four of
// its cycles whether lanes read the same bytes or not, which was 85% of the forward pass with B and C
// stored twice over, as pairs, and sums left through it; now they are paired in registers, and sums over
// the quads of states go by exchanges that halve the values a lane holds.  Neighbouring lanes hold their
// pairs of channels in opposite order, so that the first exchange needs no selection.
//
// The tokens are cut into segments, as many as fill the machine.  k_ssm_state walks every segment from
// a state of zero; k_ssm_carry goes over the segments in order and leaves the state that enters each;
// k_ssm_out or k_ssm_grad walk the segments again from there.  One segment needs the last alone.
// The backward pass keeps the state at the start of every tile: the one that k_ssm_state makes from
// zero, plus what enters the segment times exp(A sum d), so no third walk is needed; inside a
// tile the states are formed forwards, kept for two tokens at a time, and used backwards.
//
// Sequences may begin and end anywhere: a tile has a mask of the tokens that begin one (there the state
// is loaded) and of those that end one (there it is stored).  Tokens of no sequence are staged as
// d = u = g = 0, which changes no state and adds to no sum.
//
// Bound by issue: a token of 32 channels of 16 states takes 83 instructions in k_ssm_state, 124 in k_ssm_out and
// about 370 in k_ssm_grad, of which a packed one holds the issue for nearly two cycles.  16 are exponentials, at 32 a
// cycle and SM (measured), which alone would take 115 us of a walk over 65536 x 1024 x 16.  Measured there, bf16
// with gate: 224 + 14 + 322 us; gradients of 16384 x 2048 x 16: 224 + 15 + 614 + 15 us.
#include <algorithm>

#include "adj_lin.cuh"
#include "adj_profile.cuh"
#include "adj_seq.cuh"

namespace adj {
namespace {

constexpr int WPB = 4;                  // warps of a block, side by side in channels (1 for short prompts)
constexpr int G = 4;                    // tokens of a group, walked without a branch

// SWAP: neighbouring quads of states hold their channels in opposite order
template <int N_, int NP_, bool SWAP_>
struct Tile {
    static constexpr int N = N_, NP = NP_;
    static constexpr bool SWAP = SWAP_ && NP > 1;
    static constexpr int NQ = N / 4, CQ = 32 / NQ;                  // quads of states; groups of channels
    static constexpr int RC = 2 * NP, CW = RC * CQ;                 // channels of a thread, of a warp
    static constexpr int TT = 512 / CW < 4 ? 4 : 512 / CW > 16 ? 16 : 512 / CW;
    static constexpr int QR = CW / 4;                               // quads of channels in a token's row
    static constexpr int QPL = TT * QR < 32 ? 1 : TT * QR / 32;     // of a tile, a lane
    static constexpr int X = TT * CW, S = TT * N;                   // floats of a tile of channels, of B or C
    static constexpr int MPL = (S / 8 + 31) / 32;                   // a lane's vectors of eight of B or C
    static constexpr int OUT = RC > NQ ? RC / NQ : 1;               // a lane's values of a sum over states
};
constexpr int tile_tokens(int N, int np) { return 512 / (256 * np / N) < 4 ? 4 : 512 / (256 * np / N) > 16 ? 16 : 512 / (256 * np / N); }
constexpr int warp_channels(int N, int np) { return 256 * np / N; }

// four states of a thread's channels: [state][pair of channels]
template <class K>
struct States {
    pair_t v[4][K::NP];
    __device__ __forceinline__ void fill(float x) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int k = 0; k < K::NP; ++k) v[n][k] = pk(x, x);
    }
};

__device__ __forceinline__ ulonglong2 lds2(const float *p) { return *reinterpret_cast<const ulonglong2 *>(p); }
__device__ __forceinline__ pair_t lds1(const float *p) { return *reinterpret_cast<const pair_t *>(p); }
__device__ __forceinline__ void put4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ float4 get4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ pair_t twice(float x) { return pk(x, x); }
__device__ __forceinline__ pair_t shfl2(pair_t v, int d) {
    float x, y;
    upk(v, x, y);
    return pk(__shfl_xor_sync(~0u, x, d), __shfl_xor_sync(~0u, y, d));
}

// A warp's place: its channels, segment and lanes
template <class K>
struct Lane {
    int lane, nq, cq, warp, c0;         // c0: the warp's first channel
    int64_t seg, col;                   // segment, block of channels
    int64_t t0, t1;                     // the segment's tokens
    int lo, hi;                         // those that belong to sequences, counted from t0
    bool in;                            // this thread's channels exist
    __device__ Lane(const SsmArgs &a, int64_t block, int64_t cols) {
        lane = threadIdx.x & 31;
        warp = threadIdx.x >> 5;
        nq = lane % K::NQ;
        cq = lane / K::NQ;
        seg = block / cols;
        col = block - seg * cols;
        c0 = int(col * (blockDim.x >> 5) + warp) * K::CW;
        in = c0 + cq * K::RC < a.P;
        t0 = seg * a.seglen;
        t1 = min(t0 + a.seglen, a.q.rows);
        lo = 0;
        hi = int(t1 - t0);
        if (a.q.off) {
            lo = int(max(t0, a.q.at(0)) - t0);
            hi = int(max(t0, min(t1, a.q.at(a.q.B))) - t0);
        }
    }
    // first of the two channels of pair p, inside the warp's
    __device__ __forceinline__ int pair(int p) const {
        if (K::NP == 2) return cq * 4 + 2 * (p ^ (K::SWAP ? nq & 1 : 0));
        return cq * 2;
    }
    // a row [CW] of shared memory: this thread's pairs
    __device__ __forceinline__ void row(pair_t (&v)[K::NP], const float *p) const {
        if (K::NP == 2 && !K::SWAP) {
            const ulonglong2 x = lds2(p + pair(0));
            v[0] = x.x;
            v[K::NP - 1] = x.y;
        } else {
#pragma unroll
            for (int k = 0; k < K::NP; ++k) v[k] = lds1(p + pair(k));
        }
    }
    // four states of a row [N] of B or C
    __device__ __forceinline__ void maps(float (&v)[4], const float *p) const {
        const float4 x = get4(p + nq * 4);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    }
    // this thread's part of entry i of an array [.][P][N]
    __device__ __forceinline__ void load(States<K> &s, const SsmArgs &a, const float *base, int64_t i) const {
        const float *p = base + (i * a.P + c0) * K::N + nq * 4;
#pragma unroll
        for (int k = 0; k < K::NP; ++k) {
            const float4 x = in ? get4(p + pair(k) * K::N) : f4(0.f), y = in ? get4(p + (pair(k) + 1) * K::N) : f4(0.f);
            s.v[0][k] = pk(x.x, y.x);
            s.v[1][k] = pk(x.y, y.y);
            s.v[2][k] = pk(x.z, y.z);
            s.v[3][k] = pk(x.w, y.w);
        }
    }
    __device__ __forceinline__ void store(const States<K> &s, const SsmArgs &a, float *base, int64_t i) const {
        if (!in) return;
        float *p = base + (i * a.P + c0) * K::N + nq * 4;
#pragma unroll
        for (int k = 0; k < K::NP; ++k) {
            float4 x, y;
            upk(s.v[0][k], x.x, y.x);
            upk(s.v[1][k], x.y, y.y);
            upk(s.v[2][k], x.z, y.z);
            upk(s.v[3][k], x.w, y.w);
            put4(p + pair(k) * K::N, x);
            put4(p + (pair(k) + 1) * K::N, y);
        }
    }
    // a value a channel, [.][P]: written by the first quad of states
    __device__ __forceinline__ void store(const pair_t (&v)[K::NP], const SsmArgs &a, float *base, int64_t i) const {
        if (!in || nq != 0) return;
#pragma unroll
        for (int k = 0; k < K::NP; ++k) *reinterpret_cast<pair_t *>(base + i * a.P + c0 + pair(k)) = v[k];
    }
    // Sums over the quads of states of a value a channel: OUT of them a lane, from channel sums_at() of a row on;
    // lanes that hold() write them.
    __device__ __forceinline__ void sums(pair_t (&v)[K::NP], float (&o)[K::OUT]) const {
        constexpr int NQ = K::NQ;
        int m = 1;
        pair_t two = v[0];
        if (K::NP == 2) {
            two = add2(v[0], shfl2(v[K::NP - 1], 1));
            m = 2;
        }
        float x, y;
        upk(two, x, y);
        if (m >= NQ) {
            o[0] = x;
            o[K::OUT - 1] = K::OUT > 1 ? y : x;
            return;
        }
        const bool b = nq & m;
        float one = (b ? y : x) + __shfl_xor_sync(~0u, b ? x : y, m);
        for (m *= 2; m < NQ; m *= 2) one += __shfl_xor_sync(~0u, one, m);
        o[0] = one;
    }
    __device__ __forceinline__ int sums_at() const {
        if (K::NP == 2) return cq * 4 + 2 * (nq & 1) + (K::NQ > 2 ? nq >> 1 & 1 : 0);
        return cq * 2 + (nq & 1);
    }
    __device__ __forceinline__ bool hold() const { return nq < K::RC; }
    __device__ __forceinline__ void put_sums(float *row, const float (&o)[K::OUT]) const {
        float *p = row + sums_at();
        if (K::OUT == 2) *reinterpret_cast<float2 *>(p) = make_float2(o[0], o[K::OUT - 1]);
        else if (hold()) *p = o[0];
    }
};

// The sequences of a tile's tokens, bit i (lane i) for token i
struct Marks {
    int64_t b, begin, end;              // a sequence met before: most tiles lie inside it
    uint32_t first, last;
    int64_t seq;                        // of this lane's token
    __device__ Marks() : b(-1), begin(0), end(0) {}
    // forwards: the sequence of the last token is remembered, else that of the first
    template <int TT, class L>
    __device__ void at(const Seqs &q, const L &l, int64_t t, bool forwards) {
        if (b >= 0 && begin <= t && t + TT <= end) {
            first = begin == t ? 1u : 0u;
            last = end == t + TT ? 1u << (TT - 1) : 0u;
            seq = b;
            return;
        }
        const int lane = threadIdx.x & 31, i = int(t - l.t0) + lane;
        const int64_t x = t + lane;
        int64_t s = lane < TT && i >= l.lo && i < l.hi ? q.find(x) : -1, s0 = 0, s1 = 0;
        if (s >= 0) {
            s0 = q.begin(s);
            s1 = q.end(s);
        }
        first = __ballot_sync(~0u, s >= 0 && s0 == x);
        last = __ballot_sync(~0u, s >= 0 && s1 == x + 1);
        const uint32_t any = __ballot_sync(~0u, s >= 0);
        seq = s >= 0 ? s : 0;
        if (any) {
            const int k = forwards ? 31 - __clz(any) : __ffs(any) - 1;
            b = __shfl_sync(~0u, s, k);
            begin = __shfl_sync(~0u, s0, k);
            end = __shfl_sync(~0u, s1, k);
        }
    }
    __device__ __forceinline__ int64_t of(int i) const { return __shfl_sync(~0u, seq, i); }
};

// What a lane stages and finishes: quad j of channels is of token tok(j), always the same channels
template <class T, class K>
struct Mine {
    int row, cl, c;                     // cl: channel inside the warp's, c: in the array
    bool in;
    float4 bias, D;
    __device__ Mine(const SsmArgs &a, const Lane<K> &l) {
        row = l.lane / K::QR;
        cl = l.lane % K::QR * 4;
        c = l.c0 + cl;
        in = c < a.P && row < K::TT;
        bias = a.bias && in ? __ldg(reinterpret_cast<const float4 *>(a.bias + c)) : f4(0.f);
        D = a.D && in ? __ldg(reinterpret_cast<const float4 *>(a.D + c)) : f4(0.f);
    }
    __device__ __forceinline__ int tok(int j) const { return row + 32 / K::QR * j; }
    __device__ __forceinline__ bool staged() const { return row < K::TT; }
    // the tile's tokens that belong to sequences: from.. below to, counted from its first
    int from, to;
    __device__ __forceinline__ void at(const Lane<K> &l, int64_t t) {
        const int i = int(t - l.t0);
        from = max(l.lo - i, 0);
        to = min(l.hi - i, K::TT);
    }
    __device__ __forceinline__ bool ok(int j) const { return in && tok(j) >= from && tok(j) < to; }
    __device__ __forceinline__ void load(Raw4<T> (&r)[K::QPL], const void *p, int64_t ld, int64_t t) const {
        const T *q = static_cast<const T *>(p) + (t + row) * ld + c;
        const int64_t step = 32 / K::QR * ld;
#pragma unroll
        for (int j = 0; j < K::QPL; ++j) {
            if (ok(j)) r[j].load(q + j * step);
            else r[j].zero();
        }
    }
    // quad j of row tok(j) of an array [.][P] with this pitch
    __device__ __forceinline__ T *out(void *p, int64_t ld, int64_t t, int j) const {
        return static_cast<T *>(p) + (t + row) * ld + c + j * (32 / K::QR * ld);
    }
};

__device__ __forceinline__ float4 softplus4(float4 v) {
    float4 d;
    upk(softplus_2(v.x, v.y), d.x, d.y);
    upk(softplus_2(v.z, v.w), d.z, d.w);
    return d;
}

// steps and inputs of a tile: d and u = d x (zeros where there is no token)
template <class T, class K>
__device__ __forceinline__ void stage_steps(const Mine<T, K> &v, const Raw4<T> (&rx)[K::QPL], const Raw4<T> (&rdt)[K::QPL],
                                            float *ds, float *us) {
    if (!v.staged()) return;
#pragma unroll
    for (int j = 0; j < K::QPL; ++j) {
        const float4 d = v.ok(j) ? softplus4(rdt[j].get() + v.bias) : f4(0.f);
        put4(ds + v.tok(j) * K::CW + v.cl, d);
        put4(us + v.tok(j) * K::CW + v.cl, d * rx[j].get());
    }
}

// the cotangent g of v: go, times z sigmoid(z) with a gate
template <class T, class K>
__device__ __forceinline__ void stage_cotangent(const SsmArgs &a, const Mine<T, K> &v, const Raw4<T> (&rg)[K::QPL],
                                                const Raw4<T> (&rz)[K::QPL], float *gs) {
    if (!v.staged()) return;
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

// B or C of a tile
template <class T, class K>
struct Maps {
    Raw8<T> r[K::MPL];
    __device__ __forceinline__ void load(const void *p, int64_t ld, const Lane<K> &l, const Mine<T, K> &v, int64_t t) {
#pragma unroll
        for (int j = 0; j < K::MPL; ++j) {
            const int i = l.lane + 32 * j, tok = i / (K::N / 8), n = i % (K::N / 8) * 8;
            if (tok >= v.from && tok < v.to) r[j].load(static_cast<const T *>(p) + (t + tok) * ld + n);
            else r[j].zero();
        }
    }
    __device__ __forceinline__ void stage(const Lane<K> &l, float *s) const {
#pragma unroll
        for (int j = 0; j < K::MPL; ++j) {
            const int i = l.lane + 32 * j;
            float x[8];
            r[j].get(x);
            if (i < K::S / 8) {
                put4(s + i * 8, make_float4(x[0], x[1], x[2], x[3]));
                put4(s + i * 8 + 4, make_float4(x[4], x[5], x[6], x[7]));
            }
        }
    }
};

// The exponential unit's results lie low by 2e-8 on average where the exponent is near zero (measured over
// 0 to -1; 0.3 to 0.8 units of the last place at worst either way).  States that last for a
// thousand tokens would show it, so exponents are raised by that much in the multiply-add that forms them.
constexpr float EXP_UP = 2.5e-8f;

template <class K>
__device__ __forceinline__ States<K> decays(const SsmArgs &a, const Lane<K> &l) {
    States<K> A;
    l.load(A, a, a.A, 0);
    const pair_t e = twice(SEQ_LOG2E);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int k = 0; k < K::NP; ++k) A.v[n][k] = mul2(A.v[n][k], e);
    return A;
}

// what a thread reads of a token to advance its states: its channels' steps and inputs, its states' B
template <class K>
struct Token {
    pair_t d[K::NP], u[K::NP];
    float B[4];
    __device__ __forceinline__ void load(const float *ds, const float *us, const float *Bs, const Lane<K> &l, int i) {
        l.row(d, ds + i * K::CW);
        l.row(u, us + i * K::CW);
        l.maps(B, Bs + i * K::N);
    }
};

// h = exp(d A) h + u B for one token
template <bool KEEP, class K>
__device__ __forceinline__ void advance(const States<K> &A, States<K> &h, States<K> *keep, const Token<K> &k) {
    const pair_t up = twice(EXP_UP);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const pair_t B = twice(k.B[n]);
#pragma unroll
        for (int c = 0; c < K::NP; ++c) {
            const pair_t e = exp2_2(fma2(k.d[c], A.v[n][c], up));
            if (KEEP) keep->v[n][c] = e;
            h.v[n][c] = fma2(e, h.v[n][c], mul2(k.u[c], B));
        }
    }
}

// the state before a sequence's first token
template <class K>
__device__ __forceinline__ void begin_sequence(const SsmArgs &a, const Lane<K> &l, int64_t b, States<K> &h) {
    if (a.s0) l.load(h, a, a.s0, b);
    else h.fill(0.f);
}

// ---------------------------------------------------------------- segments from a state of zero
template <class K, bool BWD>
constexpr int state_floats() { return (BWD ? 3 : 2) * K::X + (BWD ? 2 : 1) * K::S; }

template <class T, int N, bool BWD>
__global__ __launch_bounds__(32 * WPB, 3) void k_ssm_state(const SsmArgs a, int64_t cols) {
    typedef Tile<N, 2, false> K;
    extern __shared__ __align__(16) float sm[];
    const Lane<K> l(a, blockIdx.x, cols);
    Mine<T, K> v(a, l);
    float *ds = sm + l.warp * state_floats<K, BWD>(), *us = ds + K::X, *Bs = us + K::X;
    float *Cs = Bs + K::S, *gs = Cs + K::S;                         // BWD
    const States<K> A = decays<K>(a, l);
    States<K> h, P, m;
    h.fill(0.f);
    P.fill(1.f);
    m.fill(0.f);
    pair_t sum[K::NP];
#pragma unroll
    for (int k = 0; k < K::NP; ++k) sum[k] = twice(0.f);
    bool fresh = false;                                             // a sequence has begun in this segment
    Marks mk;
    Raw4<T> rx[K::QPL], rdt[K::QPL];
    Maps<T, K> rB;
    auto fetch = [&](int64_t t) {
        v.at(l, t);
        v.load(rx, a.x, a.ldx, t);
        v.load(rdt, a.dt, a.lddt, t);
        rB.load(a.Bm, a.ldB, l, v, t);
    };
    fetch(l.t0);
    auto steps = [&](float *p, int64_t i) {                         // [.][P]: the sums of steps
        pair_t s[K::NP];
#pragma unroll
        for (int k = 0; k < K::NP; ++k) s[k] = fresh ? twice(-1.f) : sum[k];
        l.store(s, a, p, i);
    };
    for (int64_t t = l.t0; t < l.t1; t += K::TT) {
        if (BWD) {
            const int64_t tile = t / K::TT;
            l.store(h, a, a.tile, tile);
            steps(a.tstep, tile);
        }
        mk.at<K::TT>(a.q, l, t, true);
        __syncwarp();
        stage_steps<T, K>(v, rx, rdt, ds, us);
        rB.stage(l, Bs);
        if (BWD) {
            Raw4<T> rg[K::QPL], rz[K::QPL];
            Maps<T, K> rC;
            v.load(rg, a.go, a.ldy, t);
            if (a.z) v.load(rz, a.z, a.ldz, t);
            rC.load(a.Cm, a.ldC, l, v, t);
            stage_cotangent<T, K>(a, v, rg, rz, gs);
            rC.stage(l, Cs);
        }
        __syncwarp();
        fetch(t + K::TT);
        auto walk = [&](auto events, int i0) {
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const int i = i0 + j;
                Token<K> k;
                k.load(ds, us, Bs, l, i);
                if (events && (mk.first >> i & 1u)) {
                    begin_sequence(a, l, mk.of(i), h);
                    fresh = true;
                }
#pragma unroll
                for (int c = 0; c < K::NP; ++c) sum[c] = add2(sum[c], k.d[c]);
                States<K> e;
                advance<BWD>(A, h, &e, k);
                if (BWD && !(events && fresh)) {
                    pair_t g[K::NP];
                    float C[4];
                    l.row(g, gs + i * K::CW);
                    l.maps(C, Cs + i * N);
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int c = 0; c < K::NP; ++c) {
                            P.v[n][c] = mul2(P.v[n][c], e.v[n][c]);
                            m.v[n][c] = fma2(P.v[n][c], mul2(g[c], twice(C[n])), m.v[n][c]);
                        }
                    if (events && a.ds1 && (mk.last >> i & 1u)) {
                        States<K> s;
                        l.load(s, a, a.ds1, mk.of(i));
#pragma unroll
                        for (int n = 0; n < 4; ++n)
#pragma unroll
                            for (int c = 0; c < K::NP; ++c) m.v[n][c] = fma2(P.v[n][c], s.v[n][c], m.v[n][c]);
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
    l.store(h, a, a.seg, l.seg);
    steps(a.step, l.seg);
    if (BWD) l.store(m, a, a.adj, l.seg);
}

// Over the segments in order: seg becomes the state that enters each; blockIdx.y 1: adj, from the right.
__global__ __launch_bounds__(128) void k_ssm_carry(const SsmArgs a) {
    const int64_t i = int64_t(blockIdx.x) * 128 + threadIdx.x, n = int64_t(a.P) * a.N / 4;
    if (i >= n) return;
    const bool right = blockIdx.y != 0;
    const int p = int(i / (a.N / 4));
    const float4 A = f4(SEQ_LOG2E) * __ldg(reinterpret_cast<const float4 *>(a.A) + i);
    float4 *x = reinterpret_cast<float4 *>(right ? a.adj : a.seg) + i, cur = f4(0.f);
    constexpr int U = 16;
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
template <class K>
constexpr int out_floats() { return 3 * K::X + 2 * K::S; }

template <class T, int N, int NP>
__global__ __launch_bounds__(32 * WPB, 3) void k_ssm_out(const SsmArgs a, int64_t cols) {
    typedef Tile<N, NP, true> K;
    extern __shared__ __align__(16) float sm[];
    const int64_t work = a.nseg * cols;
    if (int64_t(blockIdx.x) >= work) {
        pass_through(a, a.s1, a.s0, blockIdx.x - work, gridDim.x - work);
        return;
    }
    const Lane<K> l(a, blockIdx.x, cols);
    Mine<T, K> v(a, l);
    float *ds = sm + l.warp * out_floats<K>(), *us = ds + K::X, *ys = us + K::X, *Bs = ys + K::X, *Cs = Bs + K::S;
    const States<K> A = decays<K>(a, l);
    States<K> h;
    h.fill(0.f);
    if (a.nseg > 1) l.load(h, a, a.seg, l.seg);
    Marks mk;
    Raw4<T> rx[K::QPL], rdt[K::QPL], rz[K::QPL], cx[K::QPL];
    Maps<T, K> rB, rC;
    auto fetch = [&](int64_t t) {
        v.at(l, t);
        v.load(rx, a.x, a.ldx, t);
        v.load(rdt, a.dt, a.lddt, t);
        rB.load(a.Bm, a.ldB, l, v, t);
        rC.load(a.Cm, a.ldC, l, v, t);
    };
    fetch(l.t0);
    for (int64_t t = l.t0; t < l.t1; t += K::TT) {
        v.at(l, t);
        mk.at<K::TT>(a.q, l, t, true);
        __syncwarp();
        stage_steps<T, K>(v, rx, rdt, ds, us);
        rB.stage(l, Bs);
        rC.stage(l, Cs);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < K::QPL; ++j) cx[j] = rx[j];
        if (a.z) v.load(rz, a.z, a.ldz, t);
        fetch(t + K::TT);
        // the sums of a group stay in registers until its end: a store to shared memory would hold up
        // the next token's loads
        auto walk = [&](auto events, int i0) {
            float o[G][K::OUT];
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const int i = i0 + j;
                Token<K> k;
                float C[4];
                k.load(ds, us, Bs, l, i);
                l.maps(C, Cs + i * N);
                if (events && (mk.first >> i & 1u)) begin_sequence(a, l, mk.of(i), h);
                advance<false>(A, h, &h, k);
                pair_t y[K::NP];
#pragma unroll
                for (int c = 0; c < K::NP; ++c) {
                    y[c] = mul2(twice(C[0]), h.v[0][c]);
#pragma unroll
                    for (int n = 1; n < 4; ++n) y[c] = fma2(twice(C[n]), h.v[n][c], y[c]);
                }
                l.sums(y, o[j]);
                if (events && a.s1 && (mk.last >> i & 1u)) {
                    const int64_t b = mk.of(i);
                    l.store(h, a, a.s1, b);
                }
            }
#pragma unroll
            for (int j = 0; j < G; ++j) l.put_sums(ys + (i0 + j) * K::CW, o[j]);
        };
#pragma unroll 1
        for (int i = 0; i < K::TT; i += G) {
            if ((mk.first | mk.last) >> i & ((1u << G) - 1)) walk(std::true_type(), i);
            else walk(std::false_type(), i);
        }
        __syncwarp();
        v.at(l, t);
#pragma unroll
        for (int j = 0; j < K::QPL; ++j) {
            if (!v.ok(j)) continue;
            float4 y = fma4(v.D, cx[j].get(), get4(ys + v.tok(j) * K::CW + v.cl));
            if (a.z) {
                const float4 z = rz[j].get();
                y = y * (z * sigmoid4(z));
            }
            st4(v.out(a.y, a.ldy, t, j), y);
        }
    }
}

// ---------------------------------------------------------------- gradients
template <int N>
struct GradSm {                         // floats of a warp's part
    typedef Tile<N, 2, true> K;
    // tokens of a group, whose states and decays stay in registers: four spill (300 bytes; 672 us against 653 for
    // 16384 x 2048 x 16 when this was chosen), but with 64 states the room for those of every second token is not there
    static constexpr int GB = N == 64 ? 4 : 2;
    static constexpr int CK = K::TT / GB * 512;                     // states at every GB-th token, [.][4][32] x 4
    static constexpr int SUM = K::TT * 2 * N;                       // dB and dC of a tile over the warp's channels
    static constexpr int ALL = 4 * K::X + 2 * K::S + CK + SUM;
};

template <class T, int N>
__global__ __launch_bounds__(32 * WPB, 2) void k_ssm_grad(const SsmArgs a, int64_t cols) {
    typedef Tile<N, 2, true> K;
    typedef GradSm<N> M;
    constexpr int NP = K::NP, GB = M::GB, RN = K::CQ == 2 ? 4 : K::CQ == 4 ? 2 : 1;
    extern __shared__ __align__(16) float sm[];
    const int64_t work = a.nseg * cols;
    if (int64_t(blockIdx.x) >= work) {
        pass_through(a, a.ds0, a.ds1, blockIdx.x - work, gridDim.x - work);
        return;
    }
    const Lane<K> l(a, blockIdx.x, cols);
    Mine<T, K> v(a, l);
    float *ds = sm + l.warp * M::ALL, *us = ds + K::X, *gs = us + K::X, *ms = gs + K::X, *Bs = ms + K::X, *Cs = Bs + K::S;
    float *ck = Cs + K::S, *ws = ck + M::CK;
    const States<K> A = decays<K>(a, l);
    States<K> e, dA;                                                // e: what reaches the state before
    l.load(e, a, a.adj, l.seg);
    dA.fill(0.f);
    float4 dD = f4(0.f), db = f4(0.f);
    Marks mk;
    const int tiles = int((l.t1 - l.t0 + K::TT - 1) / K::TT);
    for (int ti = tiles - 1; ti >= 0; --ti) {
        const int64_t t = l.t0 + int64_t(ti) * K::TT, tile = t / K::TT;
        mk.at<K::TT>(a.q, l, t, false);
        // the state before the tile
        States<K> h;
        {
            Raw4<T> rx[K::QPL], rdt[K::QPL], rg[K::QPL], rz[K::QPL];
            Maps<T, K> rB, rC;
            States<K> in;
            pair_t s[NP];
            l.load(in, a, a.seg, l.seg);
#pragma unroll
            for (int k = 0; k < NP; ++k)
                s[k] = l.in ? *reinterpret_cast<const pair_t *>(a.tstep + tile * a.P + l.c0 + l.pair(k)) : twice(-1.f);
            v.at(l, t);
            v.load(rx, a.x, a.ldx, t);
            v.load(rdt, a.dt, a.lddt, t);
            v.load(rg, a.go, a.ldy, t);
            if (a.z) v.load(rz, a.z, a.ldz, t);
            rB.load(a.Bm, a.ldB, l, v, t);
            rC.load(a.Cm, a.ldC, l, v, t);
            l.load(h, a, a.tile, tile);
            __syncwarp();
            stage_steps<T, K>(v, rx, rdt, ds, us);
            stage_cotangent<T, K>(a, v, rg, rz, gs);
            rB.stage(l, Bs);
            rC.stage(l, Cs);
            float s0, s1;
            upk(s[0], s0, s1);
            if (!(s0 < 0.f)) {                                      // a NaN is its own channel's alone
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int k = 0; k < NP; ++k) h.v[n][k] = fma2(exp2_2(mul2(s[k], A.v[n][k])), in.v[n][k], h.v[n][k]);
            }
            __syncwarp();
        }
        auto keep = [&](int g, const States<K> &x) {
#pragma unroll
            for (int n = 0; n < 4; ++n)
                *reinterpret_cast<ulonglong2 *>(ck + ((g * 4 + n) * 32 + l.lane) * 4) = make_ulonglong2(x.v[n][0], x.v[n][1]);
        };
        keep(0, h);
#pragma unroll 1
        for (int g = 1; g < K::TT / GB; ++g) {
#pragma unroll
            for (int j = 0; j < GB; ++j) {
                const int i = (g - 1) * GB + j;
                Token<K> k;
                k.load(ds, us, Bs, l, i);
                if (mk.first >> i & 1u) begin_sequence(a, l, mk.of(i), h);
                advance<false>(A, h, &h, k);
            }
            keep(g, h);
        }
        auto group = [&](auto events, int g) {
            States<K> hp[GB], ea[GB];                               // the state before each token, its decay
            float o[GB][3][K::OUT], r[GB][RN];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const ulonglong2 x = lds2(ck + ((g * 4 + n) * 32 + l.lane) * 4);
                hp[0].v[n][0] = x.x;
                hp[0].v[n][1] = x.y;
            }
#pragma unroll
            for (int j = 0; j < GB; ++j) {
                const int i = g * GB + j;
                Token<K> k;
                k.load(ds, us, Bs, l, i);
                if (events && (mk.first >> i & 1u)) begin_sequence(a, l, mk.of(i), hp[j]);
                if (j + 1 < GB) {
                    hp[j + 1] = hp[j];
                    advance<true>(A, hp[j + 1], &ea[j], k);
                } else {
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int c = 0; c < NP; ++c) ea[j].v[n][c] = exp2_2(fma2(k.d[c], A.v[n][c], twice(EXP_UP)));
                }
            }
#pragma unroll
            for (int j = GB - 1; j >= 0; --j) {
                const int i = g * GB + j;
                Token<K> k;
                pair_t gg[NP];
                float C[4];
                k.load(ds, us, Bs, l, i);
                l.row(gg, gs + i * K::CW);
                l.maps(C, Cs + i * N);
                if (events && (mk.last >> i & 1u)) {
                    const int64_t b = mk.of(i);
                    if (a.ds1) l.load(e, a, a.ds1, b);
                    else e.fill(0.f);
                }
                const pair_t zero = twice(0.f);
                pair_t vv[NP], mb[NP], sa[NP];
#pragma unroll
                for (int c = 0; c < NP; ++c) vv[c] = mb[c] = sa[c] = zero;
                float dB[4], dC[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    pair_t xb = zero, xc = zero;
                    const pair_t Bn = twice(k.B[n]), Cn = twice(C[n]);
#pragma unroll
                    for (int c = 0; c < NP; ++c) {
                        // the state after the token: the next one's, but behind the group and where another sequence begins
                        const pair_t hn = events || j == GB - 1 ? fma2(ea[j].v[n][c], hp[j].v[n][c], mul2(k.u[c], Bn)) : hp[(j + 1) % GB].v[n][c];
                        const pair_t m = fma2(gg[c], Cn, e.v[n][c]);
                        vv[c] = fma2(Cn, hn, vv[c]);
                        xc = fma2(gg[c], hn, xc);
                        xb = fma2(k.u[c], m, xb);
                        mb[c] = fma2(m, Bn, mb[c]);
                        e.v[n][c] = mul2(ea[j].v[n][c], m);
                        const pair_t w = mul2(e.v[n][c], hp[j].v[n][c]);
                        dA.v[n][c] = fma2(w, k.d[c], dA.v[n][c]);
                        sa[c] = fma2(w, A.v[n][c], sa[c]);
                    }
                    float x, y;
                    upk(xb, x, y);
                    dB[n] = x + y;
                    upk(xc, x, y);
                    dC[n] = x + y;
                }
                if (events && (mk.first >> i & 1u)) {
                    const int64_t b = mk.of(i);
                    if (a.ds0) l.store(e, a, a.ds0, b);
                    e.fill(0.f);
                }
                // Sums over states, and of dB and dC over the groups of channels: half of the lanes keep the one,
                // half the other, and so on
                l.sums(mb, o[j][0]);
                l.sums(sa, o[j][1]);
                l.sums(vv, o[j][2]);
                float q[4];
                const bool odd = l.cq & 1, b2 = l.cq & 2, b4 = l.cq & 4;
#pragma unroll
                for (int n = 0; n < 4; ++n) q[n] = (odd ? dC[n] : dB[n]) + __shfl_xor_sync(~0u, odd ? dB[n] : dC[n], K::NQ);
                if (K::CQ == 2) {
#pragma unroll
                    for (int n = 0; n < 4; ++n) r[j][n % RN] = q[n];
                } else {
                    const float r0 = (b2 ? q[2] : q[0]) + __shfl_xor_sync(~0u, b2 ? q[0] : q[2], 2 * K::NQ & 31);
                    const float r1 = (b2 ? q[3] : q[1]) + __shfl_xor_sync(~0u, b2 ? q[1] : q[3], 2 * K::NQ & 31);
                    if (K::CQ == 4) {
                        r[j][0] = r0;
                        r[j][1 % RN] = r1;
                    } else {
                        r[j][0] = (b4 ? r1 : r0) + __shfl_xor_sync(~0u, b4 ? r0 : r1, 4 * K::NQ & 31);
                        if (K::CQ == 16) r[j][0] += __shfl_xor_sync(~0u, r[j][0], 8 * K::NQ & 31);
                    }
                }
            }
            // To shared memory when the group is done, so that no store holds up a token's loads: m B, and over what is
            // done with, A e h (u's rows) and v (g's)
            __syncwarp();
#pragma unroll
            for (int j = 0; j < GB; ++j) {
                const int i = g * GB + j;
                l.put_sums(ms + i * K::CW, o[j][0]);
                l.put_sums(us + i * K::CW, o[j][1]);
                l.put_sums(gs + i * K::CW, o[j][2]);
                float *to = ws + i * 2 * N + (l.cq & 1 ? N : 0) + l.nq * 4;
                if (K::CQ == 2) put4(to, make_float4(r[j][0], r[j][1 % RN], r[j][2 % RN], r[j][3 % RN]));
                else if (K::CQ == 4) *reinterpret_cast<float2 *>(to + (l.cq & 2)) = make_float2(r[j][0], r[j][1 % RN]);
                else if (l.cq < 8) to[(l.cq & 2) + (l.cq >> 2)] = r[j][0];
            }
        };
#pragma unroll 1
        for (int g = K::TT / GB - 1; g >= 0; --g) {
            // the token behind a group may begin another sequence: that only touches its own state
            if ((mk.first | mk.last) >> (g * GB) & ((1u << GB) - 1)) group(std::true_type(), g);
            else group(std::false_type(), g);
        }
        __syncwarp();
        // the tile's gradients of what each channel reads
        {
            Raw4<T> rx[K::QPL], rdt[K::QPL], rz[K::QPL], rg[K::QPL];
            v.load(rx, a.x, a.ldx, t);
            v.load(rdt, a.dt, a.lddt, t);
            v.load(rg, a.go, a.ldy, t);
            if (a.z) v.load(rz, a.z, a.ldz, t);
#pragma unroll
            for (int j = 0; j < K::QPL; ++j) {
                if (!v.ok(j)) continue;
                const int sh = v.tok(j) * K::CW + v.cl;
                const float4 x = rx[j].get(), raw = rdt[j].get() + v.bias, mb = get4(ms + sh);
                float4 g = rg[j].get();
                if (a.z) {
                    // v z s: its derivative for z is v s (1 + z (1 - s))
                    const float4 z = rz[j].get(), s = sigmoid4(z), val = fma4(v.D, x, get4(gs + sh));
                    st4(v.out(a.dz, a.ldz, t, j), g * val * s * fma4(z, f4(1.f) - s, f4(1.f)));
                    g = g * (z * s);
                }
                const float4 ddt = fma4(x, mb, f4(SEQ_LN2) * get4(us + sh)) * sigmoid4(raw);
                st4(v.out(a.dx, a.ldx, t, j), fma4(get4(ds + sh), mb, v.D * g));
                st4(v.out(a.ddt, a.lddt, t, j), ddt);
                dD = fma4(g, x, dD);
                db = db + ddt;
            }
        }
        // dB and dC over the block's warps
        __syncthreads();
        for (int x = threadIdx.x; x < K::TT * N / 2; x += 32 * WPB) {
            const int tok = x / (N / 2), q = x % (N / 2) * 4;
            const float *p = sm + (M::ALL - M::SUM) + tok * 2 * N + q;
            float4 s = get4(p);
#pragma unroll
            for (int w = 1; w < WPB; ++w) s = s + get4(p + w * M::ALL);
            if (t + tok < l.t1) put4(a.bc + ((l.col * a.q.rows + t + tok) * 2 * N + q), s);
        }
        __syncthreads();
    }
    float *par = a.par + l.seg * a.P * (N + 2);
    l.store(dA, a, par, 0);
#pragma unroll
    for (int w = K::QR; w < 32; w <<= 1) {
        auto join = [&](float4 &x) {
            x = x + make_float4(__shfl_xor_sync(~0u, x.x, w), __shfl_xor_sync(~0u, x.y, w), __shfl_xor_sync(~0u, x.z, w),
                                __shfl_xor_sync(~0u, x.w, w));
        };
        join(dD);
        join(db);
    }
    if (l.lane < K::QR && v.in) {
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
// The state is read and written once.  256 sequences of 2048 x 16 bf16 (34 MB of states): 11.4 us where the pool stays in
// L2 between calls, 13.9 with twelve pools by turns, 20.7 behind a write over all of L2, which has to leave it first;
// the copy bandwidth gives 10.5.  Blocks of 128, not 256: 20.7 us against 22.7 in the last case; all blocks together are
// three turns of the machine, and nothing is in flight between two of them.
template <class T, int N>
__global__ __launch_bounds__(128) void k_ssm_step(const SsmArgs a, float *state, int64_t n_slots, const int32_t *slots) {
    constexpr int NQ = N / 4, K = NQ < 4 ? NQ : 4;
    const int64_t i = int64_t(blockIdx.x) * 128 + threadIdx.x, per = int64_t(a.P) / K * NQ, b = i / per;
    if (b >= a.q.B) return;                                         // whole groups of NQ lanes
    const int r = int(i - b * per), nq = r % NQ, c0 = r / NQ * K, k0 = nq % K, p = c0 + k0;
    const uint32_t group = ((1u << NQ) - 1) << (threadIdx.x & 31 & ~(NQ - 1));
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

// Two channels a thread, not four, and one segment, for a prompt so short that its walk is a matter of latency, unless
// its channels fill the SMs by themselves.  The border, 2048 x 16 bf16, us so and with four channels and segments
// of 64 tokens: 64 tokens 8.2 and 11.9, 128 14.0 and 23.7, 192 19.9 and 24.3, 256 25.3 and 24.3, 384 36.8 and 24.7;
// 2048 x 64: 192 tokens 24.4 and 29.8, 256 31.5 and 30.1, 384 45.6 and 38.2; 8192 x 16: 256 27.2 and 31.6, 384 39.2
// and 40.0.
bool brief(const SsmArgs &a) { return a.q.rows <= 256 && seq_div(a.P, warp_channels(a.N, 2)) < 608; }
int64_t columns(const SsmArgs &a, bool bwd) {
    return bwd ? seq_div(a.P, WPB * warp_channels(a.N, 2)) : brief(a) ? seq_div(a.P, warp_channels(a.N, 1))
                                                                     : seq_div(a.P, WPB * warp_channels(a.N, 2));
}
// blocks that look for sequences without tokens: only packed ones may have any, or all of them have none
int64_t lookers(const SsmArgs &a, const float *out) {
    return out && a.q.B && (a.q.off || a.q.rows == 0) ? std::min<int64_t>(a.q.B, 152) : 0;
}

template <auto Kern>
cudaError_t go(KernelId id, int64_t blocks, int warps, size_t floats, cudaStream_t st, const SsmArgs &a, int64_t cols) {
    const cudaError_t e = allow_smem<Kern>();
    if (e != cudaSuccess) return e;
    ProfScope p(id, st);
    Kern<<<unsigned(blocks), 32 * warps, warps * floats * sizeof(float), st>>>(a, cols);
    return cudaGetLastError();
}

cudaError_t carry(const SsmArgs &a, int dirs, cudaStream_t st) {
    ProfScope p(K_SSM_CARRY, st);
    k_ssm_carry<<<dim3(unsigned(seq_div(int64_t(a.P) * a.N / 4, 128)), dirs), 128, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t ssm_plan(SsmArgs &a, bool bwd, void *base) {
    const int64_t tt = tile_tokens(a.N, 2), cols = columns(a, bwd), tiles = seq_div(a.q.rows, tt);
    // whole turns of the machine: 3 blocks an SM, and backwards twice that, three turns of k_ssm_grad's 2 blocks; 64
    // tokens a segment at least (two tiles backwards: 2048 x 512 x 16 take 52 us so, 65 with one and 60 with four).
    // A short prompt stays in one segment, as its walk costs less than two more launches.
    const int64_t want = std::max<int64_t>(1, 152 * (bwd ? 6 : 3) / cols);
    const int64_t per = !bwd && brief(a) ? std::max<int64_t>(tiles, 1) : std::max<int64_t>(bwd ? 2 : 64 / tt, seq_div(tiles, want));
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
    const int64_t cols = columns(a, false), look = lookers(a, a.s1);
    return pick(a.N, bf16, [&](auto t, auto n) {
        typedef decltype(t) T;
        constexpr int N = decltype(n)::value;
        typedef Tile<N, 2, true> K;
        if (a.nseg > 1) {
            LIN_CUDA((go<k_ssm_state<T, N, false>>(K_SSM_STATE, a.nseg * cols, WPB, state_floats<K, false>(), st, a, cols)));
            LIN_CUDA(carry(a, 1, st));
        }
        if (a.nseg * cols + look == 0) return cudaSuccess;
        if (brief(a)) return go<k_ssm_out<T, N, 1>>(K_SSM_OUT, a.nseg * cols + look, 1, out_floats<Tile<N, 1, true>>(), st, a, cols);
        return go<k_ssm_out<T, N, 2>>(K_SSM_OUT, a.nseg * cols + look, WPB, out_floats<K>(), st, a, cols);
    });
}

cudaError_t launch_ssm_bwd(const SsmArgs &a, bool bf16, cudaStream_t st) {
    const int64_t cols = columns(a, true), look = lookers(a, a.ds0);
    return pick(a.N, bf16, [&](auto t, auto n) {
        typedef decltype(t) T;
        constexpr int N = decltype(n)::value;
        typedef Tile<N, 2, false> K;
        if (a.nseg) {
            LIN_CUDA((go<k_ssm_state<T, N, true>>(K_SSM_STATE, a.nseg * cols, WPB, state_floats<K, true>(), st, a, cols)));
            LIN_CUDA(carry(a, 2, st));
        }
        if (a.nseg * cols + look)
            LIN_CUDA((go<k_ssm_grad<T, N>>(K_SSM_GRAD, a.nseg * cols + look, WPB, GradSm<N>::ALL, st, a, cols)));
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
        k_ssm_step<T, N><<<unsigned(seq_div(a.q.B * (a.P / std::min(4, N / 4)) * (N / 4), 128)), 128, 0, st>>>(a, state, n_slots, slots);
        return cudaGetLastError();
    });
}

}  // namespace adj
