// adj_lin_tc.cu -- linear attention with a decay for each head on the tensor cores: the chunked
// forward and backward passes for bf16 storage.  adj_lin.cu states the formulas.
//
// Chunks of 128 tokens: every product of a chunk is one tcgen05 accumulator of 128 rows.
//     A  = Q K^T               (tokens x tokens)     exact operands
//     O1 = Q S                 (tokens x Dv)         S as a sum of two bf16
//     O2 = P V                 (tokens x Dv)         P = A . D as a sum of two bf16, in tensor memory
//     U  = (l K)^T V           (Dk x Dv)             l K as a sum of three bf16 where the state is
//                                                    a result, of two where it meets bf16 next
//     o  = scale (f O1 + O2),  S <- f_last S + U     S in fp32 registers
// with the decays D, f, l of adj_lin.cu.  Three parts hold l K to fp32, because errors in a state that is
// a result stay.  With S in one part o was off by 1.70e-3 (relative, 2-norm) over the long prompt below
// and by 2.0e-3 to 2.4e-3 where little but the state is read, for the 1.66e-3 of its own rounding; the
// second part costs that prompt 832 us for 763, and 1 to 6% where heads are smaller.
//
// One block walks the chunks of a segment of one head's tokens.  When there are fewer heads
// than SMs, the tokens of a head are cut into segments: k_lin_tc_state sums up each segment's own
// contribution, k_lin_scan joins them to the states that enter the segments, and the segments run
// in parallel; k and v are then read twice.
#include <algorithm>

#include "adj_lin.cuh"
#include "adj_profile.cuh"
#include "adj_tc5.cuh"

namespace adj {
namespace {

using namespace tc5;

constexpr int TCH = LIN_TC_CHUNK;       // tokens of a chunk
// Warps of a block: sixteen computing warps (four groups of four; a group covers the 128 lanes
// of tensor memory, a warp the lanes of its number modulo four), and one warp each that issues
// products, copies in, prepares the decays, and copies out.
constexpr int CG = 4, CW = 4 * CG;
constexpr int W_MMA = CW, W_TMA = CW + 1, W_AUX = CW + 2, W_OUT = CW + 3;
constexpr int TC_BLOCK = (CW + 4) * 32;

// The decays of one chunk, by blocks of 32 tokens.  In powers of two, with G_t the sum of the
// log decays from the chunk's start to t and E_b its value at block b's last token:
//   x[t] = G_t - E_b (b the block of t), E as hi + lo; r counts new starts
//   wb[t] = 2^(E_b - G_t): from t to its block's end, zero across a new start
//   wa[t] = 2^(G_t - E_{b-1}): from the end of the block before to t, zero across a new start (kept
//           beside this where it is used)
//   last[b]: from block b's end to the chunk's end; start[b]: from before the chunk to block b's
//           start, start[4]: over the chunk
// A decay between blocks is a product of such factors, each at most 1; only pairs inside one
// block take an exponential each.  x is hundreds to thousands where strong decays follow t in its
// block, and rounded to fp32 there (2e-4 of a decay at most): good enough for outputs of bf16
// alone.  Fp32 states and gradients take first() from wa, and pairs of a block from x with what its
// rounding lost.
struct alignas(16) ChunkDecay {
    float x[TCH], wb[TCH];
    uint8_t r[TCH];
    float Ehi[4], Elo[4], last[4];
    int re[4];
    float start[5];
    int n_cut;

    __device__ __forceinline__ float first(int t) const {
        return r[t] == 0 ? fast_exp2((Ehi[t >> 5] + Elo[t >> 5]) + x[t]) : 0.f;
    }
    __device__ __forceinline__ float first(int t, const float *wa) const { return wa[t] * start[t >> 5]; }
    __device__ __forceinline__ float to_end(int t) const { return wb[t] * last[t >> 5]; }
    __device__ __forceinline__ float total() const { return start[4]; }

    // by one whole warp: this lane's four tokens of a chunk (tokens past len have decay 1) ...
    static __device__ __forceinline__ float4 fetch(const float *g, int64_t pitch, int len) {
        const int t = (threadIdx.x & 31) * 4;
        return make_float4(t < len ? __ldg(g + t * pitch) : 0.f, t + 1 < len ? __ldg(g + (t + 1) * pitch) : 0.f,
                           t + 2 < len ? __ldg(g + (t + 2) * pitch) : 0.f, t + 3 < len ? __ldg(g + (t + 3) * pitch) : 0.f);
    }
    // ... and their decays; the chunk's sum of logarithms is returned
    // wa (may be null, and x itself): as above; xl (may be null): what the rounding of x lost
    __device__ Sum2 fill(float4 own, float *wa = nullptr, float *xl = nullptr) {
        const int lane = threadIdx.x & 31;
        const float v[4] = {own.x, own.y, own.z, own.w};
        Sum2 s[4], sum{0.f, 0.f};
        int c[4], cnt = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const bool cut = v[u] < LIN_RESET;
            const float x = cut ? 0.f : v[u];
            sum = sum + Sum2::log2_of(x);
            cnt += cut;
            s[u] = sum;
            c[u] = cnt;
        }
        Sum2 run = sum;
        int rc = cnt;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const Sum2 p = run.up(d);
            const int q = __shfl_up_sync(~0u, rc, d);
            if (lane >= d) {
                run = p + run;
                rc += q;
            }
        }
        const Sum2 E = run.from(lane | 7), Eall = run.from(31);
        const int reb = __shfl_sync(~0u, rc, lane | 7), rall = __shfl_sync(~0u, rc, 31);
        Sum2 before = run.up(1);
        if (lane == 0) before = Sum2{0.f, 0.f};
        const int cb = rc - cnt;
        float xs[4], ls[4], ws[4];
        uint32_t rs = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const Sum2 d = (before + s[u]) - E;
            xs[u] = d.value();
            ls[u] = d.lo - (xs[u] - d.hi);
            ws[u] = cb + c[u] == reb ? fast_exp2(-xs[u]) : 0.f;
            rs |= uint32_t(cb + c[u]) << (8 * u);
        }
        reinterpret_cast<float4 *>(x)[lane] = make_float4(xs[0], xs[1], xs[2], xs[3]);
        reinterpret_cast<float4 *>(wb)[lane] = make_float4(ws[0], ws[1], ws[2], ws[3]);
        reinterpret_cast<uint32_t *>(r)[lane] = rs;
        if (xl) reinterpret_cast<float4 *>(xl)[lane] = make_float4(ls[0], ls[1], ls[2], ls[3]);
        if (wa) {
            Sum2 P = run.from((lane & 24) - 1);
            int rp = __shfl_sync(~0u, rc, (lane & 24) - 1);
            if (lane < 8) {
                P = Sum2{0.f, 0.f};
                rp = 0;
            }
            float w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) w[u] = cb + c[u] == rp ? fast_exp2(((before + s[u]) - P).value()) : 0.f;
            reinterpret_cast<float4 *>(wa)[lane] = make_float4(w[0], w[1], w[2], w[3]);
        }
        if ((lane & 7) == 7) {
            const int b = lane >> 3;
            Ehi[b] = E.hi;
            Elo[b] = E.lo;
            re[b] = reb;
            last[b] = reb == rall ? fast_exp2((Eall - E).value()) : 0.f;
            start[b + 1] = reb == 0 ? fast_exp2(E.value()) : 0.f;
        }
        if (lane == 0) {
            start[0] = 1.f;
            n_cut = rall;
        }
        return Eall;
    }
};

struct FwdMaps {
    CUtensorMap q, k, v, o;
};
struct StateMaps {              // of one direction
    CUtensorMap x, y, hi, lo;   // hi, lo: the kept states
};
struct BothMaps {
    StateMaps dir[2];
};

struct Wait {
    uint64_t *bar;
    volatile int *abort;
    unsigned *status;
    // the n-th completion of barrier i
    __device__ __forceinline__ bool operator()(int i, int64_t n) const {
        return mbar_wait(smem_u32(bar + i), uint32_t(n & 1), abort, status);
    }
};
template <int N>
struct Ctl {
    uint64_t bar[N];
    uint32_t tmem;
    int abort;
};

// 8 values of row r (unit u) of a tile
__device__ __forceinline__ void put8(uint32_t tile, uint32_t panel, int r, int u, const float *v) {
    sts(tile + unit_at(r, u, panel), make_uint4(pack(v[0], v[1]), pack(v[2], v[3]), pack(v[4], v[5]), pack(v[6], v[7])));
}

// Row r of a tile times w as a sum of three bf16 (24 bits): the first in place, the others into
// tiles of their own; units u0 .. u1.
__device__ __forceinline__ void scale_row(uint32_t t0, uint32_t t1, uint32_t t2, uint32_t panel, int r, int u0, int u1,
                                          float w) {
#pragma unroll 2
    for (int u = u0; u < u1; ++u) {
        const uint32_t at = unit_at(r, u, panel);
        uint4 x = lds(t0 + at);
        if (w == 0.f) x = make_uint4(0u, 0u, 0u, 0u);    // drops a value whatever it is
        const uint32_t in[4] = {x.x, x.y, x.z, x.w};
        uint32_t h[4], l[4], ll[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a = lo_f(in[i]) * w, b = hi_f(in[i]) * w;
            h[i] = pack_top(a, b);
            a -= top(a);
            b -= top(b);
            l[i] = pack_top(a, b);
            ll[i] = pack_top(a - top(a), b - top(b));
        }
        sts(t0 + at, make_uint4(h[0], h[1], h[2], h[3]));
        sts(t1 + at, make_uint4(l[0], l[1], l[2], l[3]));
        sts(t2 + at, make_uint4(ll[0], ll[1], ll[2], ll[3]));
    }
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// The same in two parts (2^-17 of a value), three instructions for a pair of values: with
// w = w1 + w2 in bf16, x w1 has 16 bits, so h = bf16(x w1) and its remainder are exact, and x w2
// joins the remainder.
__device__ __forceinline__ void scale_row2(uint32_t t0, uint32_t t1, uint32_t panel, int r, int u0, int u1, float w) {
    const uint32_t w1 = pack(w, w);
    const float rest = w - lo_f(w1);
    const uint32_t w2 = pack(rest, rest);
#pragma unroll 4
    for (int u = u0; u < u1; ++u) {
        const uint32_t at = unit_at(r, u, panel);
        uint4 x = lds(t0 + at);
        if (w == 0.f) x = make_uint4(0u, 0u, 0u, 0u);
        const uint32_t in[4] = {x.x, x.y, x.z, x.w};
        uint32_t h[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] = mul2(in[i], w1);
            l[i] = fma2(in[i], w2, fma2(in[i], w1, h[i] ^ 0x80008000u));
        }
        sts(t0 + at, make_uint4(h[0], h[1], h[2], h[3]));
        sts(t1 + at, make_uint4(l[0], l[1], l[2], l[3]));
    }
}

// S <- tot S + U, for this thread's columns
template <int VH>
__device__ __forceinline__ void state_update(float (&S)[VH], uint32_t u, float tot) {
#pragma unroll
    for (int c = 0; c < VH; c += 16) {
        float x[16];
        ld16(u + c, x);
        if (tot == 0.f) {               // a new start drops the state whatever it holds
#pragma unroll
            for (int e = 0; e < 16; ++e) S[c + e] = x[e];
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) S[c + e] = fmaf(tot, S[c + e], x[e]);
        }
    }
}

__device__ __forceinline__ bool all_ok(bool ok) { return __all_sync(~0u, ok); }

// A segment of one head: block (b * H + h) * nseg + seg, chunks [n0, n1).
struct Seg {
    int64_t bh, b, h, hk, n0, n1;
    int seg;
    __device__ Seg(const LinArgs &a, int nseg, int cps, int64_t block) {
        bh = block / nseg;
        seg = int(block - bh * nseg);
        b = bh / a.H;
        h = bh - b * a.H;
        hk = h / (a.H / a.Hk);
        n0 = int64_t(seg) * cps;
        n1 = n0 + cps < a.NC ? n0 + cps : a.NC;
    }
};

__device__ __forceinline__ float4 gates(const LinArgs &a, const Seg &seg, int64_t chunk) {
    const int64_t t = chunk * TCH;
    return ChunkDecay::fetch(a.g + (seg.b * a.T + t) * a.H + seg.h, a.H, int(a.T - t < TCH ? a.T - t : TCH));
}

// This thread's part of a state: row d, columns c0 .. c0 + VH.
template <int VH>
__device__ __forceinline__ void load_part(float (&S)[VH], const float *p, int d, int c0, const LinArgs &a) {
#pragma unroll
    for (int u = 0; u < VH; u += 4) {
        float4 x = f4(0.f);
        if (p && d < a.Dk && c0 + u < a.Dv) x = *reinterpret_cast<const float4 *>(p + int64_t(d) * a.Dv + c0 + u);
        S[u] = x.x; S[u + 1] = x.y; S[u + 2] = x.z; S[u + 3] = x.w;
    }
}
template <int VH>
__device__ __forceinline__ void store_part(const float (&S)[VH], float *p, int d, int c0, const LinArgs &a) {
#pragma unroll
    for (int u = 0; u < VH; u += 4)
        if (d < a.Dk && c0 + u < a.Dv)
            *reinterpret_cast<float4 *>(p + int64_t(d) * a.Dv + c0 + u) = make_float4(S[u], S[u + 1], S[u + 2], S[u + 3]);
}

// ---------------------------------------------------------------- forward
// KW, VW: Dk and Dv rounded up to 64 or 128; the columns past them are zeros (the copies fill
// them) and the store clips them.
//
// Measured, 131072 tokens x 16 heads of 128 (2.15 GB): 581 us, 0.55 of the copy bandwidth, with
// 248 us for the segments' states before it.  A block takes 5.1 us a chunk.  By count the operands of
// the products, the copies, the scaled keys, the state and the output tile move 700 KB through
// shared memory, 5,500 cycles at 128 bytes a cycle: about half of that time.  The rest is taken to be
// the chain A -> l K -> U -> S and A -> P -> O2 -> o, which one block an SM cannot fill.
// The second part of S lies where the keys of the chunk before were: their product U is what S came of.
// The S tile also takes the third part of l K, between the last read of S and the next state.
enum { F_FULL0, F_FULL1, F_EMPTY0, F_EMPTY1, F_DEC0, F_DEC1, F_A, F_PV, F_P, F_K, F_U, F_S, F_OUT, F_END, F_AR, F_COUNT = F_AR + 4 };

template <int KW, int VW>
constexpr size_t fwd_smem() {
    return 2 * size_t(2 * KW + VW) * 256 + size_t(KW) * 256 + 2 * sizeof(ChunkDecay) + sizeof(Ctl<F_COUNT>);
}

template <int KW, int VW>
__global__ __launch_bounds__(TC_BLOCK, 1) void k_lin_tc_fwd(const __grid_constant__ FwdMaps m, const LinArgs a, int nseg,
                                                            int cps, int parts, unsigned *status) {
    constexpr uint32_t STAGE = (2 * KW + VW) * 256, TILE_K = KW * 256, PANEL = TCH * 128, SPANEL = KW * 128;
    constexpr int VH = VW / CG;         // state and output columns of a thread
    constexpr uint32_t T_A = 0, T_P = T_A, T_O2 = 384;
    // O1 and U take turns: the next chunk's O1 goes where U was, as soon as the state has it
    auto T_O1 = [](int64_t n) { return n & 1 ? 256u : 128u; };
    auto T_U = [](int64_t n) { return n & 1 ? 128u : 256u; };
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t base = smem_u32(sm), S_AT = base + 2 * STAGE;
    // the second part of the state that enters chunk n: where the keys of the chunk before were
    auto S_LO = [&](int64_t n) { return base + uint32_t(~n & 1) * STAGE + TILE_K; };
    ChunkDecay *dec = reinterpret_cast<ChunkDecay *>(sm + 2 * STAGE + TILE_K);
    auto *ctl = reinterpret_cast<Ctl<F_COUNT> *>(dec + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Seg seg(a, nseg, cps, blockIdx.x);
    const int64_t N = seg.n1 - seg.n0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < F_COUNT; ++i)
            mbar_init(smem_u32(&ctl->bar[i]), i >= F_AR ? CG : i == F_P || i == F_K || i == F_S || i == F_OUT ? CW : 1);
        ctl->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == W_MMA) alloc512(&ctl->tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    const Wait wait{ctl->bar, &ctl->abort, status};
    auto bar = [&](int i) { return smem_u32(&ctl->bar[i]); };

    if (warp == W_TMA) {
        if (lane == 0) {
            int64_t n = 0;
            for (; n < N; ++n) {
                const int s = int(n & 1);
                // the last chunk's O1 has read the state's second part in this stage
                if ((n >= 2 && !wait(F_EMPTY0 + s, (n >> 1) - 1)) || (n && !wait(F_A, n - 1))) break;
                const uint32_t at = base + s * STAGE, b = bar(F_FULL0 + s);
                const int t = int((seg.n0 + n) * TCH);
                mbar_arrive_expect_tx(b, STAGE);
                for (int p = 0; p < KW / 64; ++p) load4(at + p * PANEL, &m.q, p * 64, int(seg.hk), t, int(seg.b), b);
                for (int p = 0; p < KW / 64; ++p) load4(at + TILE_K + p * PANEL, &m.k, p * 64, int(seg.hk), t, int(seg.b), b);
                for (int p = 0; p < VW / 64; ++p) load4(at + 2 * TILE_K + p * PANEL, &m.v, p * 64, int(seg.h), t, int(seg.b), b);
            }
            // nothing of an abandoned walk is in flight when the block leaves
            int quiet = 0;
            for (int64_t i = n > 2 ? n - 2 : 0; i < n; ++i) mbar_wait(bar(F_FULL0 + int(i & 1)), uint32_t((i >> 1) & 1), &quiet, status);
        }
        __syncwarp();
    } else if (warp == W_AUX) {
        // decays a chunk ahead; the outputs leave through V's tile, then the stage is free
        float4 own = gates(a, seg, seg.n0);
        bool ok = true;
        auto out = [&](int64_t n) {
            const int s = int(n & 1);
            if (!all_ok(wait(F_OUT, n))) return false;
            if (lane == 0) {
                for (int p = 0; p < VW / 64; ++p)
                    store4(&m.o, p * 64, int(seg.h), int((seg.n0 + n) * TCH), int(seg.b), base + s * STAGE + 2 * TILE_K + p * PANEL);
                bulk_commit();
                bulk_wait_read();
                mbar_arrive(bar(F_EMPTY0 + s));
            }
            __syncwarp();
            return true;
        };
        for (int64_t n = 0; ok && n < N; ++n) {
            const int s = int(n & 1);
            const float4 now = own;
            if (n + 1 < N) own = gates(a, seg, seg.n0 + n + 1);
            if (n >= 2 && !(ok = out(n - 2))) break;
            dec[s].fill(now);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(F_DEC0 + s));
        }
        for (int64_t n = N > 2 ? N - 2 : 0; ok && n < N; ++n) ok = out(n);
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    } else if (warp == W_MMA) {
        if (lane == 0) {
            // a tile of one panel read across its rows gives its columns twice; the upper lanes of that
            // product are not read
            constexpr uint32_t WIDE = KW == 64 ? 0u : PANEL;
            for (int64_t n = 0; n < N; ++n) {
                const uint32_t q = base + uint32_t(n & 1) * STAGE, k = q + TILE_K, v = k + TILE_K;
                // A goes where the last P was
                if (!wait(F_FULL0 + int(n & 1), n >> 1) || (n && !wait(F_PV, n - 1))) break;
                tc_fence_after();
                product<TCH, KW / 16, false, false>(tmem + T_A, q, PANEL, k, PANEL, false);
                if (!wait(F_S, n)) break;
                tc_fence_after();
                product<VW, KW / 16, false, true>(tmem + T_O1(n), q, PANEL, S_LO(n), SPANEL, false);
                product<VW, KW / 16, false, true>(tmem + T_O1(n), q, PANEL, S_AT, SPANEL, true);
                commit(bar(F_A));
                // F_K, F_P: also every warp has read the last chunk's O1 and O2
                if (!wait(F_K, n)) break;
                tc_fence_after();
                // the accumulator truncates: the smaller parts first, while it is small
                if (parts == 3) product<VW, TCH / 16, true, true>(tmem + T_U(n), S_AT, WIDE, v, PANEL, false);
                product<VW, TCH / 16, true, true>(tmem + T_U(n), q, WIDE, v, PANEL, parts == 3);
                product<VW, TCH / 16, true, true>(tmem + T_U(n), k, WIDE, v, PANEL, true);
                commit(bar(F_U));
                if (!wait(F_P, n)) break;
                tc_fence_after();
                product_ts<VW, TCH / 16>(tmem + T_O2, tmem + T_P, v, PANEL, false);
                product_ts<VW, TCH / 16>(tmem + T_O2, tmem + T_P + 64, v, PANEL, true);
                commit(bar(F_PV));
            }
            int quiet = 0;
            commit(bar(F_END));
            mbar_wait(bar(F_END), 0, &quiet, status);
        }
        __syncwarp();
    } else if (warp < CW) {
        const int wq = warp & 3, g = warp >> 2, i = wq * 32 + lane, c0 = g * VH;
        const uint32_t lanes = tmem + (uint32_t(wq * 32) << 16);
        auto arrive = [&](int b) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(b));
        };
        float S[VH];
        const int64_t dd = int64_t(a.Dk) * a.Dv;
        load_part<VH>(S, nseg > 1 ? a.S + int64_t(blockIdx.x) * dd : a.s0 ? a.s0 + seg.bh * dd : nullptr, i, c0, a);
        auto put_state = [&](int64_t n) {
            if (i < KW) {
                const uint32_t lo = S_LO(n);
#pragma unroll
                for (int u = 0; u < VH; u += 8) {
                    const uint32_t at = unit_at(i, (c0 + u) >> 3, SPANEL);
                    uint32_t h[4], l[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = S[u + 2 * e], y = S[u + 2 * e + 1];
                        h[e] = pack_top(x, y);
                        l[e] = pack(x - top(x), y - top(y));
                    }
                    sts(S_AT + at, make_uint4(h[0], h[1], h[2], h[3]));
                    sts(lo + at, make_uint4(l[0], l[1], l[2], l[3]));
                }
            }
            fence_proxy_async_smem();
            arrive(F_S);
        };
        put_state(0);
        for (int64_t n = 0; n < N; ++n) {
            const int s = int(n & 1);
            const uint32_t Q = base + s * STAGE, K = Q + TILE_K, V = K + TILE_K;
            const ChunkDecay &d = dec[s];
            // l K: the products of Q, K and S are done, and their tiles take its three parts.  K and the
            // decays are waited for too: A's barrier orders the products alone, not what other warps and
            // the copies have written
            if (!all_ok(wait(F_FULL0 + s, n >> 1) && wait(F_DEC0 + s, n >> 1) && wait(F_A, n))) break;
            tc_fence_after();
            if (parts == 3) scale_row(K, Q, S_AT, PANEL, i, g * (KW / 8 / CG), (g + 1) * (KW / 8 / CG), d.to_end(i));
            else scale_row2(K, Q, PANEL, i, g * (KW / 8 / CG), (g + 1) * (KW / 8 / CG), d.to_end(i));
            fence_proxy_async_smem();
            arrive(F_K);
            // P while U is formed: 8 g .. + 8 of every block of 32 columns, in place of A
            {
                const float xi = d.x[i];
                const int ri = d.r[i];
                uint32_t h[4][4], l[4][4];
                auto split = [&](int c, const float (&p)[8]) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        h[c][e] = pack_top(p[2 * e], p[2 * e + 1]);
                        l[c][e] = pack_top(p[2 * e] - top(p[2 * e]), p[2 * e + 1] - top(p[2 * e + 1]));
                    }
                };
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float A[8], w[8];
                    const int j0 = 32 * c + 8 * g;
                    if (c < wq) {
                        ld8(lanes + T_A + j0, A);
                        const float f =
                            ri == d.re[c] ? a.scale * fast_exp2((d.Ehi[wq] - d.Ehi[c]) + (d.Elo[wq] - d.Elo[c]) + xi) : 0.f;
                        *reinterpret_cast<float4 *>(w) = *reinterpret_cast<const float4 *>(d.wb + j0);
                        *reinterpret_cast<float4 *>(w + 4) = *reinterpret_cast<const float4 *>(d.wb + j0 + 4);
#pragma unroll
                        for (int e = 0; e < 8; ++e) A[e] *= w[e] * f;
                        split(c, A);
                    } else if (c == wq) {
                        ld8(lanes + T_A + j0, A);
                        *reinterpret_cast<float4 *>(w) = *reinterpret_cast<const float4 *>(d.x + j0);
                        *reinterpret_cast<float4 *>(w + 4) = *reinterpret_cast<const float4 *>(d.x + j0 + 4);
                        const uint2 rj = *reinterpret_cast<const uint2 *>(d.r + j0);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int r = int(((e < 4 ? rj.x : rj.y) >> (8 * (e & 3))) & 255u);
                            A[e] = 8 * g + e <= lane && ri == r ? A[e] * (a.scale * fast_exp2(xi - w[e])) : 0.f;
                        }
                        split(c, A);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) h[c][e] = l[c][e] = 0u;
                    }
                }
                tc_fence_before();
                arrive(F_AR + wq);
                // the warps of these lanes have read their columns
                if (!all_ok(wait(F_AR + wq, n))) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    st4(lanes + T_P + 16 * c + 4 * g, h[c][0], h[c][1], h[c][2], h[c][3]);
                    st4(lanes + T_P + 64 + 16 * c + 4 * g, l[c][0], l[c][1], l[c][2], l[c][3]);
                }
                st_wait();
                tc_fence_before();
                arrive(F_P);
            }
            if (!all_ok(wait(F_U, n))) break;
            tc_fence_after();
            state_update<VH>(S, lanes + T_U(n) + c0, d.total());
            tc_fence_before();
            put_state(n + 1);
            // the outputs, through V's tile
            const float f = d.first(i) * a.scale;
            if (!all_ok(wait(F_PV, n))) break;
            tc_fence_after();
#pragma unroll
            for (int u = 0; u < VH; u += 16) {
                float x[16], y[16];
                ld16x2(lanes + T_O1(n) + c0 + u, lanes + T_O2 + c0 + u, x, y);
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = f == 0.f ? y[e] : fmaf(f, x[e], y[e]);
                put8(V, PANEL, i, (c0 + u) >> 3, y);
                put8(V, PANEL, i, ((c0 + u) >> 3) + 1, y + 8);
            }
            tc_fence_before();
            fence_proxy_async_smem();
            arrive(F_OUT);
        }
        if (a.s1 && nseg == 1) store_part<VH>(S, a.s1 + seg.bh * dd, i, c0, a);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W_MMA) {
        tc_fence_after();
        free512(tmem);
    }
}

// ---------------------------------------------------------------- segment states
// Measured, 131072 tokens x 16 heads of 128 in 9 segments (1.07 GB): 247 us.
//
// The state that a segment's own tokens leave (zero before it): S[blockIdx.x], and the decay
// over it; in the second half of a grid for both directions, the adjoint state from q and scale go,
// walked from the last chunk back.
//
// A ring of three stages of half a chunk (64 tokens).  The warps multiply x by its decays to the
// chunk's end (two more tiles of a stage take the second and third part), the products of a
// chunk's two halves add up in one of two accumulators, and the warps fold the chunk before into
// the state meanwhile; only the state's own multiply-add is a chain.
constexpr int SH = TCH / 2, RING = 3;
enum { S_FULL, S_EMPTY = S_FULL + RING, S_K = S_EMPTY + RING, S_DEC = S_K + RING, S_DFREE = S_DEC + 2,
       S_U = S_DFREE + 2, S_UFREE = S_U + 2, S_KEPT = S_UFREE + 2, S_END, S_LEFT, S_COUNT };

template <int KW, int VW, bool KEEP>
constexpr size_t state_smem() {
    return RING * size_t(3 * KW + VW) * SH * 2 + (KEEP ? size_t(KW) * VW * 2 : 0) + 2 * sizeof(ChunkDecay) + sizeof(Ctl<S_COUNT>);
}

// Columns of a piece of a kept state's third part.
constexpr int PIECE = 32;
// KEEP: the walk starts from the state that enters the segment (a.S / a.dS, or s0 / ds1 when the
// segment is the whole head), and the state met before every chunk is kept as a sum of three bf16
// [B,H,NC,Dk,Dv], the operand of the backward pass.  The first two leave one after the other through
// one tile, the second while the next chunk is being scaled; with a tile each and a ring of two
// stages the walk waited for its copies in (all state launches of 2 x 8192 tokens x 16 heads of
// 128: 241 us so, 208 us with one tile and three stages).  The third leaves from the registers with the
// second, 32 bytes a store in a layout of its own (the same launches now: 198 us, 183 us without a
// third part, 310 us with it through the tile as well).
template <int KW, int VW, bool KEEP>
__global__ __launch_bounds__(TC_BLOCK, 1) void k_lin_tc_state(const __grid_constant__ BothMaps maps, const LinArgs a,
                                                              int nseg, int cps, unsigned *status) {
    constexpr uint32_t TILE_K = KW * SH * 2, TILE_V = VW * SH * 2, STAGE = 3 * TILE_K + TILE_V, PANEL = SH * 128;
    constexpr uint32_t TILE_S = KW * VW * 2, SPANEL = KW * 128;
    constexpr int VH = VW / CG;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t base = smem_u32(sm), KEPT = base + RING * STAGE;
    ChunkDecay *dec = reinterpret_cast<ChunkDecay *>(sm + RING * STAGE + (KEEP ? TILE_S : 0));
    auto *ctl = reinterpret_cast<Ctl<S_COUNT> *>(dec + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t per = a.B * a.H * nseg, block = blockIdx.x % per;
    const bool rev = blockIdx.x >= per;
    const StateMaps &m = maps.dir[rev];
    const Seg seg(a, nseg, cps, block);
    const int64_t N = seg.n1 - seg.n0;
    auto chunk = [&](int64_t n) { return rev ? seg.n1 - 1 - n : seg.n0 + n; };
    // no segment reads what the last one leaves: only the final state does
    if (!KEEP && seg.seg == (rev ? 0 : nseg - 1) && !(rev ? a.ds0 : a.s1)) return;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S_COUNT; ++i)
            mbar_init(smem_u32(&ctl->bar[i]), (i >= S_K && i < S_DEC) || (i >= S_DFREE && i < S_U) || (i >= S_UFREE && i <= S_KEPT) ? CW : 1);
        ctl->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == W_MMA) alloc512(&ctl->tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    const Wait wait{ctl->bar, &ctl->abort, status};
    auto bar = [&](int i) { return smem_u32(&ctl->bar[i]); };
    auto arrive = [&](int b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(b));
    };

    if (warp == W_TMA) {
        if (lane == 0) {
            int64_t h = 0, turn = 0;    // halves loaded; the ring's turn
            int s = 0;
            for (; h < 2 * N; ++h) {
                if (turn && !wait(S_EMPTY + s, turn - 1)) break;
                const uint32_t at = base + s * STAGE, b = bar(S_FULL + s);
                const int t = int(chunk(h >> 1) * TCH + (h & 1) * SH);
                mbar_arrive_expect_tx(b, TILE_K + TILE_V);
                for (int p = 0; p < KW / 64; ++p) load4(at + p * PANEL, &m.x, p * 64, int(seg.hk), t, int(seg.b), b);
                for (int p = 0; p < VW / 64; ++p) load4(at + 3 * TILE_K + p * PANEL, &m.y, p * 64, int(seg.h), t, int(seg.b), b);
                if (++s == RING) { s = 0; ++turn; }
            }
            // nothing of an abandoned walk is in flight when the block leaves
            int quiet = 0;
            for (int64_t i = h > RING ? h - RING : 0; i < h; ++i)
                mbar_wait(bar(S_FULL + int(i % RING)), uint32_t((i / RING) & 1), &quiet, status);
        }
        __syncwarp();
    } else if (warp == W_AUX) {
        Sum2 sum{0.f, 0.f};
        int cuts = 0;
        float4 own = gates(a, seg, chunk(0));
        for (int64_t n = 0; n < N; ++n) {
            const int s = int(n & 1);
            const float4 now = own;
            if (n + 1 < N) own = gates(a, seg, chunk(n + 1));
            if (n >= 2 && !all_ok(wait(S_DFREE + s, (n >> 1) - 1))) break;
            sum = sum + dec[s].fill(now, rev ? dec[s].x : nullptr);     // x itself is not read
            __syncwarp();
            cuts += dec[s].n_cut;
            if (lane == 0) mbar_arrive(bar(S_DEC + s));
        }
        if (!KEEP && lane == 0) (rev ? a.dtot : a.tot)[block] = cuts ? 0.f : fast_exp2(sum.value());
    } else if (warp == W_OUT) {
        if (KEEP && lane == 0) {
            for (int64_t k = 0; k < 2 * N; ++k) {
                if (!wait(S_KEPT, k)) break;
                for (int p = 0; p < VW / 64; ++p)
                    store3(k & 1 ? &m.lo : &m.hi, p * 64, 0, int(seg.bh * a.NC + chunk(k >> 1)), KEPT + p * SPANEL);
                bulk_commit();
                bulk_wait_read();
                mbar_arrive(bar(S_LEFT));
            }
            bulk_wait_all();
        }
        __syncwarp();
    } else if (warp == W_MMA) {
        if (lane == 0) {
            constexpr uint32_t WIDE = KW == 64 ? 0u : PANEL;
            int64_t turn = 0;
            int s = 0;
            for (int64_t h = 0; h < 2 * N; ++h) {
                const int64_t n = h >> 1;
                const int u = int(n & 1);
                if (!wait(S_FULL + s, turn) || !wait(S_K + s, turn)) break;
                if (!(h & 1) && n >= 2 && !wait(S_UFREE + u, (n >> 1) - 1)) break;
                tc_fence_after();
                const uint32_t at = base + s * STAGE, y = at + 3 * TILE_K, d = tmem + u * 128;
                // the accumulator truncates: the smaller parts first
#pragma unroll
                for (int p = 2; p >= 0; --p)
                    product<VW, SH / 16, true, true>(d, at + p * TILE_K, WIDE, y, PANEL, p < 2 || (h & 1));
                commit(bar(S_EMPTY + s));
                if (h & 1) commit(bar(S_U + u));
                if (++s == RING) { s = 0; ++turn; }
            }
            int quiet = 0;
            commit(bar(S_END));
            mbar_wait(bar(S_END), 0, &quiet, status);
        }
        __syncwarp();
    } else if (warp < CW) {
        // x times its decays: row r of the half, an eighth of the units
        constexpr int UQ = KW / 8 / 8;
        const int r = threadIdx.x & 63, q = threadIdx.x >> 6;
        const int wq = warp & 3, g = warp >> 2, i = wq * 32 + lane, c0 = g * VH;
        const uint32_t lanes = tmem + (uint32_t(wq * 32) << 16);
        float S[VH];
        const int64_t dd = int64_t(a.Dk) * a.Dv;
        const float *init = rev ? a.ds1 : a.s0;
        load_part<VH>(S, !KEEP ? nullptr : nseg > 1 ? (rev ? a.dS : a.S) + block * dd : init ? init + seg.bh * dd : nullptr,
                      i, c0, a);
        // the first (k even) or second part of the state; k counts the parts
        // and the third with it
        auto keep = [&](int64_t k) {
            if (!KEEP) return true;
            if (k && !all_ok(wait(S_LEFT, k - 1))) return false;
            if (i < KW) {
                const int pieces = lin_pieces(a.Dv);
                __nv_bfloat16 *third = (rev ? a.z3 : a.s3) + ((seg.bh * a.NC + chunk(k >> 1)) * pieces * a.Dk + i) * PIECE;
                uint4 before = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int u = 0; u < VH; u += 8) {
                    uint32_t h[4], t[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = S[u + 2 * e], y = S[u + 2 * e + 1];
                        h[e] = pack(x, y);
                        if (k & 1) {
                            x -= lo_f(h[e]);
                            y -= hi_f(h[e]);
                            h[e] = pack(x, y);
                            t[e] = pack_top(x - lo_f(h[e]), y - hi_f(h[e]));
                        }
                    }
                    sts(KEPT + unit_at(i, (c0 + u) >> 3, SPANEL), make_uint4(h[0], h[1], h[2], h[3]));
                    if (k & 1) {
                        const uint4 now = make_uint4(t[0], t[1], t[2], t[3]);
                        const int e = c0 + u - 8;
                        if ((u & 8) && i < a.Dk && e / PIECE < pieces) stg32(third + e / PIECE * a.Dk * PIECE + e % PIECE, before, now);
                        before = now;
                    }
                }
            }
            fence_proxy_async_smem();
            arrive(S_KEPT);
            return true;
        };
        auto fold = [&](int64_t n, float tot) {
            const int u = int(n & 1);
            if (!all_ok(wait(S_U + u, n >> 1))) return false;
            tc_fence_after();
            state_update<VH>(S, lanes + u * 128 + c0, tot);
            tc_fence_before();
            arrive(S_UFREE + u);
            return true;
        };
        bool ok = true;
        float tot = 0.f;
        int64_t turn = 0;
        int s = 0;
        for (int64_t n = 0; ok && n < N; ++n) {
            const int e = int(n & 1);
            if (!(ok = all_ok(wait(S_DEC + e, n >> 1)))) break;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                if (!(ok = all_ok(wait(S_FULL + s, turn)))) break;
                const uint32_t at = base + s * STAGE;
                scale_row(at, at + TILE_K, at + 2 * TILE_K, PANEL, r, q * UQ, (q + 1) * UQ,
                          rev ? dec[e].first(h * SH + r, dec[e].x) * a.scale : dec[e].to_end(h * SH + r));
                fence_proxy_async_smem();
                arrive(S_K + s);
                if (++s == RING) { s = 0; ++turn; }
                if (h == 0 && n && !(ok = keep(2 * n - 1))) break;
            }
            const float now = dec[e].total();
            if (!ok) break;
            arrive(S_DFREE + e);
            if (n && !(ok = fold(n - 1, tot))) break;
            if (!(ok = keep(2 * n))) break;
            tot = now;
        }
        if (ok && keep(2 * N - 1)) fold(N - 1, tot);
        if (!KEEP) store_part<VH>(S, (rev ? a.dS : a.S) + block * dd, i, c0, a);
        else if (rev && a.ds0 && seg.seg == 0) store_part<VH>(S, a.ds0 + seg.bh * dd, i, c0, a);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W_MMA) {
        tc_fence_after();
        free512(tmem);
    }
}

// ---------------------------------------------------------------- gradients of a chunk
// One chunk of one head at a time, any order: the states around it are there (k_lin_tc_state).
// With W = go, R = scale D . (W V^T) and P = scale D . (Q K^T) (tokens x tokens, lower triangle):
//     dq = R K + scale f (W S^T)        dk = R^T Q + l (V Z^T)        dv = P^T W + l (K Z)
// R, and R^T and P^T from products of their own (V W^T, K Q^T: a transpose is dearer than eight
// instructions), are sums of two bf16 that take the columns of the fp32 values they come from, so that
// no warp waits for another's reads.  dg does not go through them: its sums over
// W_ij = R_ij (q_i . k_j) are taken from the fp32 accumulators, by rows from R and by columns from R^T,
// and S and Z come as sums of three bf16 (dv takes two of Z's).  The accumulators drop what is below
// their last bit: smaller parts are multiplied first.
// The third parts come in pieces of 32 columns beside the tiles.  Without them the training batch below
// takes 389 us for 433, and dg is off by 1e-6 to 4.5e-6 for 0.8e-7 to 4.9e-7.
// Measured, 2 x 8192 tokens x 16 heads of 128 (2048 chunks): 225 us, 16 us a chunk and SM; the
// states before it 200 us in two launches.  Bound by the chain of a chunk: its products and four
// passes of the registers, each waiting for the one before.
// Tensor memory: four accumulators of 128 columns; R^T and P^T lie where their products were.
// The outputs leave through tiles whose last product is done: dq through S's, dk through Q's, dv
// through Z's (fp32 parts of shared heads are stored by the lanes), so that the next task's Q, K, V
// and W come in while dv is formed.  The decays are a task ahead.
struct GradMaps {
    CUtensorMap q, k, v, w, shi, slo, s3, zhi, zlo, z3, dq, dk, dv;
};
struct GradSums {
    float r[CG][TCH], f[CG][TCH], l[CG][TCH];   // W: rows less columns; reads of S; leavings to Z
    float zs[CW];
};
enum { G_IN, G_S, G_Z, G_DEC0, G_DEC1, G_X1, G_R, G_D1, G_X2, G_RT, G_D2, G_D3, G_E1, G_E2, G_SC, G_DONE, G_DG,
       G_OQ, G_OK, G_OV, G_SFREE, G_QFREE, G_LEFT, G_END, G_T, G_TFREE = G_T + 3, G_COUNT = G_TFREE + 3 };

template <int KW, int VW>
constexpr size_t grad_smem() {
    return 2 * size_t(KW + VW) * 256 + 2 * size_t(KW) * VW * 2 + 3 * size_t(KW) * PIECE * 2 + 2 * (sizeof(ChunkDecay) + TCH * 8) + sizeof(GradSums) +
           sizeof(Ctl<G_COUNT>);
}

// 16 columns of a row to an fp32 array of 16-byte aligned rows; columns past n are left out
__device__ __forceinline__ void put16(float *p, int n, const float (&v)[16]) {
#pragma unroll
    for (int u = 0; u < 16; u += 4)
        if (u < n) *reinterpret_cast<float4 *>(p + u) = make_float4(v[u], v[u + 1], v[u + 2], v[u + 3]);
}

template <int KW, int VW>
__global__ __launch_bounds__(TC_BLOCK, 1) void k_lin_tc_grad(const __grid_constant__ GradMaps m, const LinArgs a,
                                                             int64_t tasks, unsigned *status) {
    constexpr uint32_t TILE_K = KW * 256, TILE_V = VW * 256, PANEL = TCH * 128, SPANEL = KW * 128, TILE_S = KW * VW * 2;
    constexpr int KH = KW / CG, VH = VW / CG;   // columns of a thread
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t Q = smem_u32(sm), K = Q + TILE_K, V = K + TILE_K, W = V + TILE_V, SHI = W + TILE_V, SLO = SHI + TILE_S,
                   THIRD = SLO + TILE_S;
    constexpr int PN = VW / PIECE;
    constexpr uint32_t TILE_P = KW * PIECE * 2;
    ChunkDecay *decs = reinterpret_cast<ChunkDecay *>(sm + 2 * (TILE_K + TILE_V) + 2 * TILE_S + 3 * TILE_P);
    float *was = reinterpret_cast<float *>(decs + 2);   // wa and xl of both
    GradSums &sums = *reinterpret_cast<GradSums *>(was + 4 * TCH);
    auto *ctl = reinterpret_cast<Ctl<G_COUNT> *>(&sums + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr uint32_t R0 = 0, R1 = 128, R2 = 256, R3 = 384;

    if (threadIdx.x == 0) {
        for (int i = 0; i < G_COUNT; ++i)
            mbar_init(smem_u32(&ctl->bar[i]), i == G_R || i == G_RT || (i >= G_E1 && i <= G_DONE) || (i >= G_OQ && i <= G_OV) ? CW : 1);
        ctl->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == W_MMA) alloc512(&ctl->tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    const Wait wait{ctl->bar, &ctl->abort, status};
    auto bar = [&](int i) { return smem_u32(&ctl->bar[i]); };
    auto arrive = [&](int b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(b));
    };
    // the n-th task of this block
    struct Task {
        int64_t bh, b, h, hk, n;
    };
    auto task = [&](int64_t n) {
        // below 2^31, as the map of the states wants it
        const uint32_t t = blockIdx.x + uint32_t(n) * gridDim.x, nc = uint32_t(a.NC), H = uint32_t(a.H);
        const uint32_t bh = t / nc, b = bh / H, h = bh - b * H;
        return Task{bh, b, h, h / (H / uint32_t(a.Hk)), t - bh * nc};
    };
    const int64_t N = (tasks - blockIdx.x + gridDim.x - 1) / gridDim.x;

    if (warp == W_TMA) {
        if (lane == 0) {
            int64_t n = 0;
            int in = 0, ss = 0, zz = 0;         // copies begun
            int64_t turn = 0;                   // the ring's turn
            int at = 0;
            // pieces p0 .. p1 of a state's third part, as the products with those before are done
            auto load_third = [&](const CUtensorMap *x, int p0, int p1, int z) {
                for (int p = p0; p < p1; ++p) {
                    if (turn && !wait(G_TFREE + at, turn - 1)) return false;
                    mbar_arrive_expect_tx(bar(G_T + at), TILE_P);
                    load4(THIRD + at * TILE_P, x, 0, 0, p, z, bar(G_T + at));   // past the state: zeros
                    if (++at == 3) { at = 0; ++turn; }
                }
                return true;
            };
            constexpr int PA = PN < 3 ? PN : 3;
            for (; n < N; ++n) {
                // the last task is done with the tiles: its products, and dk has left
                if (n && !(wait(G_D3, n - 1) && wait(G_QFREE, n - 1))) break;
                const Task k = task(n);
                const int t = int(k.n * TCH), z = int(k.bh * a.NC + k.n);
                mbar_arrive_expect_tx(bar(G_IN), 2 * (TILE_K + TILE_V));
                ++in;
                for (int p = 0; p < VW / 64; ++p) {
                    load4(W + p * PANEL, &m.w, p * 64, int(k.h), t, int(k.b), bar(G_IN));
                    load4(V + p * PANEL, &m.v, p * 64, int(k.h), t, int(k.b), bar(G_IN));
                }
                for (int p = 0; p < KW / 64; ++p) {
                    load4(Q + p * PANEL, &m.q, p * 64, int(k.hk), t, int(k.b), bar(G_IN));
                    load4(K + p * PANEL, &m.k, p * 64, int(k.hk), t, int(k.b), bar(G_IN));
                }
                if (!load_third(&m.s3, 0, PA, z)) break;
                if (n && !wait(G_LEFT, n - 1)) break;         // dv too
                mbar_arrive_expect_tx(bar(G_S), 2 * TILE_S);
                ++ss;
                for (int p = 0; p < VW / 64; ++p) {
                    load3(SHI + p * SPANEL, &m.shi, p * 64, 0, z, bar(G_S));
                    load3(SLO + p * SPANEL, &m.slo, p * 64, 0, z, bar(G_S));
                }
                if (!(load_third(&m.s3, PA, PN, z) && load_third(&m.z3, 0, PA, z))) break;
                // Z in S's place, once dq has left through it
                if (!wait(G_SFREE, n)) break;
                mbar_arrive_expect_tx(bar(G_Z), 2 * TILE_S);
                ++zz;
                for (int p = 0; p < VW / 64; ++p) {
                    load3(SHI + p * SPANEL, &m.zhi, p * 64, 0, z, bar(G_Z));
                    load3(SLO + p * SPANEL, &m.zlo, p * 64, 0, z, bar(G_Z));
                }
                if (!load_third(&m.z3, PA, PN, z)) break;
            }
            // nothing of an abandoned walk is in flight when the block leaves
            int quiet = 0;
            if (in) mbar_wait(bar(G_IN), uint32_t(in - 1) & 1, &quiet, status);
            if (ss) mbar_wait(bar(G_S), uint32_t(ss - 1) & 1, &quiet, status);
            if (zz) mbar_wait(bar(G_Z), uint32_t(zz - 1) & 1, &quiet, status);
            for (int i = 0; i < 3; ++i)
                if (turn + (i < at)) mbar_wait(bar(G_T + i), uint32_t(turn + (i < at) - 1) & 1, &quiet, status);
        }
        __syncwarp();
    } else if (warp == W_OUT) {
        if (lane == 0) {
            for (int64_t n = 0; n < N; ++n) {
                const Task k = task(n);
                const int t = int(k.n * TCH);
                if (!wait(G_OQ, n)) break;
                if (!a.pq) {
                    for (int p = 0; p < KW / 64; ++p) store4(&m.dq, p * 64, int(k.hk), t, int(k.b), SHI + p * PANEL);
                    bulk_commit();
                    bulk_wait_read();
                }
                mbar_arrive(bar(G_SFREE));
                if (!wait(G_OK, n)) break;
                if (!a.pq) {
                    for (int p = 0; p < KW / 64; ++p) store4(&m.dk, p * 64, int(k.hk), t, int(k.b), Q + p * PANEL);
                    bulk_commit();
                    bulk_wait_read();
                }
                mbar_arrive(bar(G_QFREE));
                if (!wait(G_OV, n)) break;
                for (int p = 0; p < VW / 64; ++p) store4(&m.dv, p * 64, int(k.h), t, int(k.b), SHI + p * PANEL);
                bulk_commit();
                bulk_wait_read();
                mbar_arrive(bar(G_LEFT));
            }
            bulk_wait_all();
        }
        __syncwarp();
    } else if (warp == W_AUX) {
        // decays a task ahead, and the sums of dg when a task is done
        auto fetch = [&](int64_t n) {
            const Task k = task(n);
            const int64_t t0 = k.n * TCH;
            return ChunkDecay::fetch(a.g + (k.b * a.T + t0) * a.H + k.h, a.H, int(a.T - t0 < TCH ? a.T - t0 : TCH));
        };
        auto fill = [&](int64_t n, float4 own) {
            decs[n & 1].fill(own, was + (n & 1) * 2 * TCH, was + (n & 1) * 2 * TCH + TCH);
            arrive(G_DEC0 + int(n & 1));
        };
        fill(0, fetch(0));
        for (int64_t n = 0; n < N; ++n) {
            const Task k = task(n);
            const int64_t t0 = k.n * TCH;
            const int len = int(a.T - t0 < TCH ? a.T - t0 : TCH);
            if (n + 1 < N) fill(n + 1, fetch(n + 1));    // its buffer's last task was done before this one
            const ChunkDecay &dec = decs[n & 1];
            if (!all_ok(wait(G_DONE, n))) break;
            float r[4], f[4], l[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int t = lane * 4 + u;
                r[u] = f[u] = l[u] = 0.f;
#pragma unroll
                for (int g = 0; g < CG; ++g) {
                    r[u] += sums.r[g][t];
                    f[u] += sums.f[g][t];
                    l[u] += sums.l[g][t];
                }
            }
            float zs = lane < CW ? sums.zs[lane] : 0.f;
#pragma unroll
            for (int d = 16; d; d >>= 1) zs += __shfl_xor_sync(~0u, zs, d);
            // suffix sums of r and f, prefix sums of l, within the lane and then across the warp
            const float lt = (l[0] + l[1]) + (l[2] + l[3]);
            r[2] += r[3]; r[1] += r[2]; r[0] += r[1];
            f[2] += f[3]; f[1] += f[2]; f[0] += f[1];
            float rr = r[0], ff = f[0], ll = lt;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const float x = __shfl_down_sync(~0u, rr, d), y = __shfl_down_sync(~0u, ff, d), z = __shfl_up_sync(~0u, ll, d);
                if (lane + d < 32) {
                    rr += x;
                    ff += y;
                }
                if (lane >= d) ll += z;
            }
            const float after_r = rr - r[0], after_f = ff - f[0];
            float across = (ll - lt) + (dec.total() == 0.f ? 0.f : dec.total() * zs);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int t = lane * 4 + u;
                const bool cut = t ? dec.r[t] != dec.r[t - 1] : dec.r[0] != 0;
                // no pair of the chunk crosses its first token
                if (t < len)
                    a.dg[(k.b * a.T + t0 + t) * a.H + k.h] = cut ? 0.f : across + (f[u] + after_f) + (t ? r[u] + after_r : 0.f);
                across += l[u];
            }
            arrive(G_DG);
        }
    } else if (warp == W_MMA) {
        if (lane == 0) {
            constexpr int KS = KW / 16, VS = VW / 16, T8 = TCH / 8;
            int64_t turn = 0;
            int at = 0;
            // R2 = x times the third part of a state
            auto thirds = [&](uint32_t x) {
                for (int p = 0; p < PN; ++p) {
                    if (!wait(G_T + at, turn)) return false;
                    tc_fence_after();
                    product32<KW>(tmem + R2, x + (p >> 1) * PANEL + (p & 1) * (PIECE * 2), THIRD + at * TILE_P, p != 0);
                    commit(bar(G_TFREE + at));
                    if (++at == 3) { at = 0; ++turn; }
                }
                return true;
            };
            for (int64_t n = 0; n < N; ++n) {
                if (!wait(G_IN, n)) break;
                tc_fence_after();
                product<TCH, VS, false, false>(tmem + R0, W, PANEL, V, PANEL, false);
                product<TCH, KS, false, false>(tmem + R1, Q, PANEL, K, PANEL, false);
                commit(bar(G_X1));
                // the accumulator truncates: the smaller parts first.  R2 has been read (dv)
                if (!((n == 0 || wait(G_DONE, n - 1)) && thirds(W) && wait(G_S, n))) break;
                tc_fence_after();
                product<KW, VS, false, false>(tmem + R2, W, PANEL, SLO, SPANEL, true);
                product<KW, VS, false, false>(tmem + R2, W, PANEL, SHI, SPANEL, true);
                if (!wait(G_R, n)) break;
                tc_fence_after();
                product_ts2<KW, T8>(tmem + R3, tmem + R0, K, PANEL);
                commit(bar(G_D1));
                product<TCH, KS, false, false>(tmem + R1, K, PANEL, Q, PANEL, false);
                if (!wait(G_D1, n)) break;              // R0 has been read
                tc_fence_after();
                product<TCH, VS, false, false>(tmem + R0, V, PANEL, W, PANEL, false);
                commit(bar(G_X2));
                if (!(wait(G_E1, n) && thirds(V) && wait(G_Z, n))) break;
                tc_fence_after();
                product<KW, VS, false, false>(tmem + R2, V, PANEL, SLO, SPANEL, true);
                product<KW, VS, false, false>(tmem + R2, V, PANEL, SHI, SPANEL, true);
                if (!wait(G_RT, n)) break;
                tc_fence_after();
                product_ts2<KW, T8>(tmem + R3, tmem + R0, Q, PANEL);
                commit(bar(G_D2));
                if (!wait(G_E2, n)) break;
                tc_fence_after();
                product<VW, KS, false, true>(tmem + R2, K, PANEL, SLO, SPANEL, false);
                product<VW, KS, false, true>(tmem + R2, K, PANEL, SHI, SPANEL, true);
                product_ts2<VW, T8>(tmem + R3, tmem + R1, W, PANEL);
                commit(bar(G_D3));
            }
            int quiet = 0;
            commit(bar(G_END));
            mbar_wait(bar(G_END), 0, &quiet, status);
        }
        __syncwarp();
    } else if (warp < CW) {
        const int wq = warp & 3, g = warp >> 2, i = wq * 32 + lane;
        const uint32_t lanes = tmem + (uint32_t(wq * 32) << 16);
        for (int64_t n = 0; n < N; ++n) {
            const Task k = task(n);
            const int64_t t0 = k.n * TCH;
            const bool live = t0 + i < a.T;
            const int64_t tok = k.b * a.T + t0 + i;
            const ChunkDecay &dec = decs[n & 1];
            const float *wa = was + (n & 1) * 2 * TCH, *xl = wa + TCH;
            // the tiles too, whose rows are read below: the products' barriers do not order the copies
            if (!all_ok(wait(G_DEC0 + int(n & 1), n >> 1) && wait(G_IN, n) && (n == 0 || wait(G_DG, n - 1)) && wait(G_X1, n)))
                break;
            tc_fence_after();
            const float xi = dec.x[i], xli = xl[i], wai = wa[i];
            const int ri = dec.r[i], j8 = 8 * g;
            // what x's rounding lost at this thread's 8 columns of its own block
            auto lost = [&](float (&w)[8]) {
                *reinterpret_cast<float4 *>(w) = *reinterpret_cast<const float4 *>(xl + 32 * wq + j8);
                *reinterpret_cast<float4 *>(w + 4) = *reinterpret_cast<const float4 *>(xl + 32 * wq + j8 + 4);
            };
            // R, 8 columns of every block of 32, and the row sums of W
            {
                float sum = 0.f;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t h[8] = {};
                    if (c > wq) {
                        st8(lanes + R0 + 32 * c + j8, h);
                        continue;
                    }
                    float x[8], y[8], w[8];
                    ld8(lanes + R0 + 32 * c + j8, x);
                    ld8(lanes + R1 + 32 * c + j8, y);
                    const float *src = (c < wq ? dec.wb : dec.x) + 32 * c + j8;
                    *reinterpret_cast<float4 *>(w) = *reinterpret_cast<const float4 *>(src);
                    *reinterpret_cast<float4 *>(w + 4) = *reinterpret_cast<const float4 *>(src + 4);
                    if (c < wq) {
                        // c < wq: the block before this row's exists
                        const int p = wq ? wq - 1 : 0;
                        const float f = dec.re[p] == dec.re[c]
                                            ? a.scale * wai * fast_exp2((dec.Ehi[p] - dec.Ehi[c]) + (dec.Elo[p] - dec.Elo[c])) : 0.f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            x[e] *= w[e] * f;
                            sum = fmaf(x[e], y[e], sum);
                        }
                    } else {
                        const uint2 rj = *reinterpret_cast<const uint2 *>(dec.r + 32 * c + j8);
                        float l[8];
                        lost(l);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int r = int(((e < 4 ? rj.x : rj.y) >> (8 * (e & 3))) & 255u);
                            x[e] = j8 + e <= lane && ri == r ? x[e] * (a.scale * fast_exp2((xi - w[e]) + (xli - l[e]))) : 0.f;
                            if (j8 + e < lane) sum = fmaf(x[e], y[e], sum);
                        }
                    }
                    split8(x, h);
                    st8(lanes + R0 + 32 * c + j8, h);
                }
                sums.r[g][i] = sum;
                st_wait();
                tc_fence_before();
                arrive(G_R);
            }
            // 8 values of row i of the state in the tiles, from column 8 u of this thread's; <Z, S> takes the
            // third part where at least 1 / 64 of it crosses the chunk
            const bool deep = dec.total() >= 1.f / 64;
            auto state8 = [&](int u, const __nv_bfloat16 *third, float (&v)[8]) {
                const int c = g * VH + 8 * u;
                const uint32_t at = i < KW ? unit_at(i, c >> 3, SPANEL) : 0u;
                const uint4 x = lds(SHI + at), y = lds(SLO + at);
                uint4 t = make_uint4(0u, 0u, 0u, 0u);
                if (deep && i < a.Dk && c < a.Dv)
                    t = __ldg(reinterpret_cast<const uint4 *>(
                        third + (((k.bh * a.NC + k.n) * lin_pieces(a.Dv) + c / PIECE) * a.Dk + i) * PIECE + c % PIECE));
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w}, ts[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[2 * e] = (lo_f(xs[e]) + lo_f(ys[e])) + lo_f(ts[e]);
                    v[2 * e + 1] = (hi_f(xs[e]) + hi_f(ys[e])) + hi_f(ts[e]);
                }
            };
            // this thread's part of S
            float S[VH / 8][8];
            if (!all_ok(wait(G_S, n))) break;
#pragma unroll
            for (int u = 0; u < VH / 8; ++u) state8(u, a.s3, S[u]);
            // dq takes S's place: every warp has its part, and W S^T is formed
            arrive(G_SC);
            auto stage = [&](uint32_t tile, int c, const float (&y)[16]) {
                put8(tile, PANEL, i, c >> 3, y);
                put8(tile, PANEL, i, (c >> 3) + 1, y + 8);
            };
            // an output of one phase: s R2 + R3, and s R2 . x with x this row's tile
            auto out = [&](float s, uint32_t tile, int c0, int W_, auto put, float *dot) {
                float d = 0.f;
#pragma unroll 1
                for (int u = 0; u < W_; u += 16) {
                    float x[16], y[16];
                    ld16x2(lanes + R2 + c0 + u, lanes + R3 + c0 + u, x, y);
                    if (dot) {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const uint4 v = lds(tile + unit_at(i, ((c0 + u) >> 3) + q, PANEL));
                            const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                d = fmaf(x[8 * q + 2 * e], lo_f(in[e]), d);
                                d = fmaf(x[8 * q + 2 * e + 1], hi_f(in[e]), d);
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) y[e] = s == 0.f ? y[e] : fmaf(s, x[e], y[e]);
                    put(c0 + u, y);
                }
                if (dot) *dot = s == 0.f ? 0.f : s * d;
            };
            // dq
            const float fi = dec.first(i, wa) * a.scale;
            if (!all_ok(wait(G_SC, n) && wait(G_D1, n))) break;
            tc_fence_after();
            out(fi, Q, g * KH, KH, [&](int c, const float (&y)[16]) {
                if (!a.pq) stage(SHI, c, y);
                else if (live) put16(a.pq + (tok * a.H + k.h) * a.Dk + c, a.Dk - c, y);
            }, &sums.f[g][i]);
            tc_fence_before();
            arrive(G_E1);
            fence_proxy_async_smem();
            arrive(G_OQ);
            // R^T and P^T: this thread's row is token j = i, its columns the later tokens
            if (!all_ok(wait(G_X2, n))) break;
            tc_fence_after();
            const float wbj = dec.wb[i];
            {
                float sum = 0.f;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t h[8] = {};
                    if (c < wq) {
                        st8(lanes + R0 + 32 * c + j8, h);
                        st8(lanes + R1 + 32 * c + j8, h);
                        continue;
                    }
                    float x[8], y[8], w[8];
                    ld8(lanes + R0 + 32 * c + j8, x);
                    ld8(lanes + R1 + 32 * c + j8, y);
                    const float *src = (c > wq ? wa : dec.x) + 32 * c + j8;
                    *reinterpret_cast<float4 *>(w) = *reinterpret_cast<const float4 *>(src);
                    *reinterpret_cast<float4 *>(w + 4) = *reinterpret_cast<const float4 *>(src + 4);
                    if (c > wq) {
                        const float f = dec.re[c - 1 < 0 ? 0 : c - 1] == dec.re[wq]
                                            ? a.scale * wbj *
                                                  fast_exp2((dec.Ehi[c - 1 < 0 ? 0 : c - 1] - dec.Ehi[wq]) +
                                                            (dec.Elo[c - 1 < 0 ? 0 : c - 1] - dec.Elo[wq]))
                                            : 0.f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float d = w[e] * f;
                            x[e] *= d;
                            sum = fmaf(x[e], y[e], sum);
                            y[e] *= d;
                        }
                    } else {
                        const uint2 rj = *reinterpret_cast<const uint2 *>(dec.r + 32 * c + j8);
                        float l[8];
                        lost(l);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int r = int(((e < 4 ? rj.x : rj.y) >> (8 * (e & 3))) & 255u);
                            const bool in = j8 + e >= lane && ri == r;
                            const float d = in ? a.scale * fast_exp2((w[e] - xi) + (l[e] - xli)) : 0.f;
                            x[e] = in ? x[e] * d : 0.f;
                            if (j8 + e > lane) sum = fmaf(x[e], y[e], sum);
                            y[e] = in ? y[e] * d : 0.f;
                        }
                    }
                    split8(x, h);
                    st8(lanes + R0 + 32 * c + j8, h);
                    split8(y, h);
                    st8(lanes + R1 + 32 * c + j8, h);
                }
                sums.r[g][i] -= sum;
                st_wait();
                tc_fence_before();
                arrive(G_RT);
            }
            // <Z, S>
            if (!all_ok(wait(G_Z, n))) break;
            {
                float d = 0.f;
#pragma unroll
                for (int u = 0; u < VH / 8; ++u) {
                    float z[8];
                    state8(u, a.z3, z);
#pragma unroll
                    for (int e = 0; e < 8; ++e) d = fmaf(z[e], S[u][e], d);
                }
                if (i >= KW) d = 0.f;
#pragma unroll
                for (int e = 16; e; e >>= 1) d += __shfl_xor_sync(~0u, d, e);
                if (lane == 0) sums.zs[warp] = d;
            }
            // dk
            const float lj = dec.to_end(i);
            if (!all_ok(wait(G_D2, n))) break;
            tc_fence_after();
            out(lj, K, g * KH, KH, [&](int c, const float (&y)[16]) {
                if (!a.pk) stage(Q, c, y);
                else if (live) put16(a.pk + (tok * a.H + k.h) * a.Dk + c, a.Dk - c, y);
            }, &sums.l[g][i]);
            tc_fence_before();
            arrive(G_E2);
            fence_proxy_async_smem();
            arrive(G_OK);
            // dv
            if (!all_ok(wait(G_D3, n))) break;
            tc_fence_after();
            out(lj, 0u, g * VH, VH, [&](int c, const float (&y)[16]) {
                stage(SHI, c, y);            // Z has been read: <Z, S> by all warps (G_E2), K Z (G_D3)
            }, static_cast<float *>(nullptr));
            tc_fence_before();
            fence_proxy_async_smem();
            arrive(G_OV);
            arrive(G_DONE);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W_MMA) {
        tc_fence_after();
        free512(tmem);
    }
}

// dirs: 1 forward, 2 both
template <int KW, int VW, bool KEEP>
cudaError_t run_states(const LinArgs &a, const LinSplit &sp, int dirs, unsigned *status, cudaStream_t st) {
    BothMaps m;
    const int64_t n = a.B * a.H * a.NC;
    bool ok = map_tokens(&m.dir[0].x, a.k, a.Dk, a.Hk, a.T, a.B, a.ldk, SH) && map_tokens(&m.dir[0].y, a.v, a.Dv, a.H, a.T, a.B, a.ldv, SH);
    if (dirs == 2)
        ok = ok && map_tokens(&m.dir[1].x, a.q, a.Dk, a.Hk, a.T, a.B, a.ldq, SH) && map_tokens(&m.dir[1].y, a.go, a.Dv, a.H, a.T, a.B, a.ldo, SH);
    if (KEEP)
        ok = ok && map_states(&m.dir[0].hi, a.shi, a.Dv, a.Dk, n, KW) && map_states(&m.dir[0].lo, a.slo, a.Dv, a.Dk, n, KW) &&
             map_states(&m.dir[1].hi, a.zhi, a.Dv, a.Dk, n, KW) && map_states(&m.dir[1].lo, a.zlo, a.Dv, a.Dk, n, KW);
    if (!ok) return cudaErrorInvalidValue;
    constexpr size_t smem = state_smem<KW, VW, KEEP>();
    LIN_CUDA((allow_smem<k_lin_tc_state<KW, VW, KEEP>>(smem)));
    ProfScope ps(K_LIN_STATE, st);
    k_lin_tc_state<KW, VW, KEEP><<<unsigned(a.B * a.H * sp.nseg * dirs), TC_BLOCK, smem, st>>>(m, a, sp.nseg, sp.cps, status);
    return cudaGetLastError();
}

template <int KW, int VW>
cudaError_t run_fwd(const LinArgs &a, const LinSplit &sp, unsigned *status, cudaStream_t st) {
    static_assert(fwd_smem<128, 128>() <= 232448 && state_smem<128, 128, false>() <= 232448 &&
                      state_smem<128, 128, true>() <= 232448, "shared memory of an SM");
    FwdMaps m;
    if (!map_tokens(&m.q, a.q, a.Dk, a.Hk, a.T, a.B, a.ldq) || !map_tokens(&m.k, a.k, a.Dk, a.Hk, a.T, a.B, a.ldk) ||
        !map_tokens(&m.v, a.v, a.Dv, a.H, a.T, a.B, a.ldv) || !map_tokens(&m.o, a.o, a.Dv, a.H, a.T, a.B, a.ldo))
        return cudaErrorInvalidValue;
    if (sp.nseg > 1) {
        LIN_CUDA((run_states<KW, VW, false>(a, sp, 1, status, st)));
        LIN_CUDA(launch_lin_scan(a, sp.nseg, 1, st));
    }
    constexpr size_t smem = fwd_smem<KW, VW>();
    LIN_CUDA((allow_smem<k_lin_tc_fwd<KW, VW>>(smem)));
    ProfScope ps(K_LIN_OUT, st);
    // the state is a result only where no segments' states were joined: otherwise it meets bf16 next
    const int parts = sp.nseg == 1 && a.s1 ? 3 : 2;
    k_lin_tc_fwd<KW, VW><<<unsigned(a.B * a.H * sp.nseg), TC_BLOCK, smem, st>>>(m, a, sp.nseg, sp.cps, parts, status);
    return cudaGetLastError();
}

template <int KW, int VW>
cudaError_t run_bwd(const LinArgs &a, const LinSplit &sp, unsigned *status, cudaStream_t st) {
    static_assert(grad_smem<128, 128>() <= 232448, "shared memory of an SM");
    GradMaps m;
    const int64_t n = a.B * a.H * a.NC;
    if (!map_tokens(&m.q, a.q, a.Dk, a.Hk, a.T, a.B, a.ldq) || !map_tokens(&m.k, a.k, a.Dk, a.Hk, a.T, a.B, a.ldk) ||
        !map_tokens(&m.v, a.v, a.Dv, a.H, a.T, a.B, a.ldv) || !map_tokens(&m.w, a.go, a.Dv, a.H, a.T, a.B, a.ldo) ||
        !map_states(&m.shi, a.shi, a.Dv, a.Dk, n, KW) || !map_states(&m.slo, a.slo, a.Dv, a.Dk, n, KW) ||
        (!a.pq && (!map_tokens(&m.dq, a.dq, a.Dk, a.Hk, a.T, a.B, a.ldq) || !map_tokens(&m.dk, a.dk, a.Dk, a.Hk, a.T, a.B, a.ldk))) ||
        !map_tokens(&m.dv, a.dv, a.Dv, a.H, a.T, a.B, a.ldv) || !map_states(&m.zhi, a.zhi, a.Dv, a.Dk, n, KW) || !map_states(&m.zlo, a.zlo, a.Dv, a.Dk, n, KW))
        return cudaErrorInvalidValue;
    const int pieces = lin_pieces(a.Dv);
    if (!map_pieces(&m.s3, a.s3, a.Dk, pieces, n, KW) || !map_pieces(&m.z3, a.z3, a.Dk, pieces, n, KW)) return cudaErrorInvalidValue;
    // the states around every chunk: by segments where the heads alone would leave SMs idle
    LinArgs b = a;
    b.s1 = b.ds0 = nullptr;
    if (sp.nseg > 1) {
        LIN_CUDA((run_states<KW, VW, false>(b, sp, 2, status, st)));
        LIN_CUDA(launch_lin_scan(b, sp.nseg, 3, st));
    }
    LIN_CUDA((run_states<KW, VW, true>(a, sp, 2, status, st)));
    constexpr size_t smem = grad_smem<KW, VW>();
    LIN_CUDA((allow_smem<k_lin_tc_grad<KW, VW>>(smem)));
    ProfScope ps(K_LIN_GRAD, st);
    k_lin_tc_grad<KW, VW><<<unsigned(std::min<int64_t>(n, 152)), TC_BLOCK, smem, st>>>(m, a, n, status);
    return cudaGetLastError();
}

}  // namespace

LinSplit lin_split(const LinArgs &a, bool bwd) {
    // the backward pass walks both directions side by side
    const int64_t heads = a.B * a.H * (bwd ? 2 : 1), NC = a.NC;
    LinSplit s{1, int(NC)};
    // One block an SM: split the tokens when that fills SMs that would stay idle; a segment is at
    // least four chunks, below which its start costs more than it saves.
    if (heads < 152 && NC >= 8) {
        int64_t n = std::min<int64_t>(152 / heads, NC / 4);
        if (n > 1) {
            s.cps = int(lin_div(NC, n));
            s.nseg = int(lin_div(NC, s.cps));
        }
    }
    return s;
}

cudaError_t launch_lin_tc_fwd(const LinArgs &a, unsigned *status, cudaStream_t st) {
    const LinSplit sp = lin_split(a, false);
    if (a.Dk <= 64) return a.Dv <= 64 ? run_fwd<64, 64>(a, sp, status, st) : run_fwd<64, 128>(a, sp, status, st);
    return a.Dv <= 64 ? run_fwd<128, 64>(a, sp, status, st) : run_fwd<128, 128>(a, sp, status, st);
}

cudaError_t launch_lin_tc_bwd(const LinArgs &a, unsigned *status, cudaStream_t st) {
    const LinSplit sp = lin_split(a, true);
    if (a.Dk <= 64) return a.Dv <= 64 ? run_bwd<64, 64>(a, sp, status, st) : run_bwd<64, 128>(a, sp, status, st);
    return a.Dv <= 64 ? run_bwd<128, 64>(a, sp, status, st) : run_bwd<128, 128>(a, sp, status, st);
}

}  // namespace adj
