// adj_lin_tc.cu -- linear attention with a decay for each head on the tensor cores: the chunked
// forward pass for bf16 storage.  adj_lin.cu states the formulas.
//
// Chunks of 128 tokens: every product of a chunk is one tcgen05 accumulator of 128 rows.
//     A  = Q K^T               (tokens x tokens)     exact operands
//     O1 = Q S                 (tokens x Dv)         S rounded to bf16
//     O2 = P V                 (tokens x Dv)         P = A . D rounded to bf16, in tensor memory
//     U  = (l K)^T V           (Dk x Dv)             l K as a sum of two bf16, 2^-17 of a value
//     o  = scale (f O1 + O2),  S <- f_last S + U     S in fp32 registers
// with the decays D, f, l of adj_lin.cu.  O1 and O2 have one rounding to bf16 each, as large as
// that of the output itself; U is held closer because the state is an fp32 result and errors
// in it stay.
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

constexpr int TCH = 128;                // tokens of a chunk
constexpr int CW = 8;                   // computing warps: two groups of four, a group covers the 128 lanes
constexpr int W_MMA = CW, W_TMA = CW + 1, W_DEC = CW + 2;
constexpr int TC_BLOCK = (CW + 3) * 32;

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The decays of one chunk, by blocks of 32 tokens.  In powers of two, with G_t the sum of the
// log decays from the chunk's start to t and E_b its value at block b's last token:
//   x[t] = G_t - E_b (b the block of t), E as hi + lo; r counts new starts
//   wb[t] = 2^(E_b - G_t): from t to its block's end, zero across a new start
//   last[b]: from block b's end to the chunk's end; total: over the chunk
// A decay between blocks is a product of such factors, each at most 1; only pairs inside one
// block take an exponential each.
struct ChunkDecay {
    float x[TCH], wb[TCH];
    uint8_t r[TCH];
    float Ehi[4], Elo[4], last[4];
    int re[4];
    float total;
    int n_cut;

    __device__ __forceinline__ float first(int t) const {
        return r[t] == 0 ? fast_exp2((Ehi[t >> 5] + Elo[t >> 5]) + x[t]) : 0.f;
    }
    __device__ __forceinline__ float to_end(int t) const { return wb[t] * last[t >> 5]; }

    // by one whole warp: g[n * pitch], n < len (tokens past len have decay 1); the chunk's sum of
    // logarithms is returned
    __device__ double fill(const float *g, int64_t pitch, int len) {
        const int lane = threadIdx.x & 31;
        double s[4], sum = 0.0;
        int c[4], cnt = 0;
        float v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = lane * 4 + u < len ? __ldg(g + (lane * 4 + u) * pitch) : 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const bool cut = v[u] < LIN_RESET;
            sum += cut ? 0.0 : double(v[u]) * 1.4426950408889634;
            cnt += cut;
            s[u] = sum;
            c[u] = cnt;
        }
        double run = sum;
        int rc = cnt;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const double p = __shfl_up_sync(~0u, run, d);
            const int q = __shfl_up_sync(~0u, rc, d);
            if (lane >= d) {
                run += p;
                rc += q;
            }
        }
        const double E = __shfl_sync(~0u, run, lane | 7), Eall = __shfl_sync(~0u, run, 31);
        const int reb = __shfl_sync(~0u, rc, lane | 7), rall = __shfl_sync(~0u, rc, 31);
        const double before = run - sum;
        const int cb = rc - cnt;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int t = lane * 4 + u;
            const float d = float((before + s[u]) - E);
            x[t] = d;
            r[t] = uint8_t(cb + c[u]);
            wb[t] = cb + c[u] == reb ? fast_exp2(-d) : 0.f;
        }
        if ((lane & 7) == 7) {
            const int b = lane >> 3;
            Ehi[b] = float(E);
            Elo[b] = float(E - double(float(E)));
            re[b] = reb;
            last[b] = reb == rall ? fast_exp2(float(Eall - E)) : 0.f;
        }
        if (lane == 0) {
            total = rall == 0 ? fast_exp2(float(Eall)) : 0.f;
            n_cut = rall;
        }
        return Eall;
    }
};

struct FwdMaps {
    CUtensorMap q, k, v, o;
};
struct StateMaps {
    CUtensorMap x, y;
};

enum { B_FULL0, B_FULL1, B_EMPTY0, B_EMPTY1, B_DEC0, B_DEC1, B_A, B_O1, B_P, B_K, B_U, B_S, B_OFREE, B_END, B_COUNT };
struct Ctl {
    uint64_t bar[B_COUNT];
    uint32_t tmem;
    int abort;
};

// Write 32 consecutive values (as bf16) of row r from column `col` on into a tile.
__device__ __forceinline__ void put32(uint32_t tile, uint32_t panel, int r, int col, const float (&v)[32]) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
        sts(tile + unit_at(r, (col >> 3) + u, panel),
            make_uint4(pack(v[8 * u], v[8 * u + 1]), pack(v[8 * u + 2], v[8 * u + 3]), pack(v[8 * u + 4], v[8 * u + 5]),
                       pack(v[8 * u + 6], v[8 * u + 7])));
}

// Row r of a tile times w, as hi + lo: hi in place, lo into the other tile; units u0 .. u1.
__device__ __forceinline__ void scale_row(uint32_t hi, uint32_t lo, uint32_t panel, int r, int u0, int u1, float w) {
#pragma unroll 4
    for (int u = u0; u < u1; ++u) {
        const uint32_t at = unit_at(r, u, panel);
        const uint4 x = lds(hi + at);
        const uint32_t in[4] = {x.x, x.y, x.z, x.w};
        uint32_t h[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = w == 0.f ? 0.f : lo_f(in[i]) * w, b = w == 0.f ? 0.f : hi_f(in[i]) * w;
            h[i] = pack(a, b);
            l[i] = pack(a - lo_f(h[i]), b - hi_f(h[i]));
        }
        sts(hi + at, make_uint4(h[0], h[1], h[2], h[3]));
        sts(lo + at, make_uint4(l[0], l[1], l[2], l[3]));
    }
}

__device__ __forceinline__ bool all_ok(bool ok) { return __all_sync(~0u, ok); }

struct Wait {
    uint64_t *bar;
    volatile int *abort;
    unsigned *status;
    __device__ __forceinline__ bool operator()(int i, int64_t n) const {
        return mbar_wait(smem_u32(bar + i), uint32_t(n & 1), abort, status);
    }
};

// A segment of one head: blockIdx.x = (b * H + h) * nseg + seg, chunks [n0, n1).
struct Seg {
    int64_t bh, b, h, hk, n0, n1;
    int seg;
    __device__ Seg(const LinArgs &a, int nseg, int cps) {
        bh = blockIdx.x / nseg;
        seg = int(blockIdx.x - bh * nseg);
        b = bh / a.H;
        h = bh - b * a.H;
        hk = h / (a.H / a.Hk);
        n0 = int64_t(seg) * cps;
        n1 = n0 + cps < a.NC ? n0 + cps : a.NC;
    }
};

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
template <int KW, int VW>
constexpr size_t fwd_smem() {
    return 2 * size_t(2 * KW + VW) * 256 + size_t(KW) * VW * 2 + 2 * sizeof(ChunkDecay) + sizeof(Ctl);
}

template <int KW, int VW>
__global__ __launch_bounds__(TC_BLOCK, 1) void k_lin_tc_fwd(const __grid_constant__ FwdMaps m, const LinArgs a, int nseg,
                                                            int cps, unsigned *status) {
    constexpr uint32_t STAGE = (2 * KW + VW) * 256, TILE_K = KW * 256, PANEL = TCH * 128, SPANEL = KW * 128;
    constexpr int VH = VW / 2;          // state and output columns of a thread
    constexpr uint32_t T_A = 0, T_U = 128, T_O1 = 256, T_O2 = 384;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t base = smem_u32(sm), S_AT = base + 2 * STAGE;
    ChunkDecay *dec = reinterpret_cast<ChunkDecay *>(sm + 2 * STAGE + KW * VW * 2);
    Ctl *ctl = reinterpret_cast<Ctl *>(dec + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Seg seg(a, nseg, cps);
    const int64_t N = seg.n1 - seg.n0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < B_COUNT; ++i)
            mbar_init(smem_u32(&ctl->bar[i]), i == B_P || i == B_K || i == B_S || i == B_OFREE ? CW : 1);
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
                if (n >= 2 && !wait(B_EMPTY0 + s, (n >> 1) - 1)) break;
                const uint32_t at = base + s * STAGE, b = bar(B_FULL0 + s);
                const int t = int((seg.n0 + n) * TCH);
                mbar_arrive_expect_tx(b, STAGE);
                for (int p = 0; p < KW / 64; ++p) load4(at + p * PANEL, &m.q, p * 64, int(seg.hk), t, int(seg.b), b);
                for (int p = 0; p < KW / 64; ++p) load4(at + TILE_K + p * PANEL, &m.k, p * 64, int(seg.hk), t, int(seg.b), b);
                for (int p = 0; p < VW / 64; ++p) load4(at + 2 * TILE_K + p * PANEL, &m.v, p * 64, int(seg.h), t, int(seg.b), b);
            }
            // nothing of an abandoned walk is in flight when the block leaves
            int quiet = 0;
            for (int64_t i = n > 2 ? n - 2 : 0; i < n; ++i) mbar_wait(bar(B_FULL0 + int(i & 1)), uint32_t((i >> 1) & 1), &quiet, status);
        }
        __syncwarp();
    } else if (warp == W_DEC) {
        for (int64_t n = 0; n < N; ++n) {
            const int s = int(n & 1);
            if (n >= 2 && !all_ok(wait(B_EMPTY0 + s, (n >> 1) - 1))) break;
            const int64_t t = (seg.n0 + n) * TCH;
            dec[s].fill(a.g + (seg.b * a.T + t) * a.H + seg.h, a.H, int(a.T - t < TCH ? a.T - t : TCH));
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_DEC0 + s));
        }
    } else if (warp == W_MMA) {
        if (lane == 0) {
            const int kd = (a.Dk + 15) >> 4;
            auto tiles = [&](int64_t n, Tile &q, Tile &k, Tile &v) {
                const uint32_t at = base + uint32_t(n & 1) * STAGE;
                q = Tile{at, PANEL, false};
                k = Tile{at + TILE_K, PANEL, false};
                v = Tile{at + 2 * TILE_K, PANEL, true};
            };
            Tile q, k, v;
            tiles(0, q, k, v);
            bool ok = wait(B_FULL0, 0);
            if (ok) {
                tc_fence_after();
                product(tmem + T_A, q, k, TCH, kd, false);
                commit(bar(B_A));
            }
            for (int64_t n = 0; ok && n < N; ++n) {
                tiles(n, q, k, v);
                ok = wait(B_S, n) && (n == 0 || wait(B_OFREE, n - 1));
                if (!ok) break;
                tc_fence_after();
                product(tmem + T_O1, q, Tile{S_AT, SPANEL, true}, VW, kd, false);
                commit(bar(B_O1));
                if (!(ok = wait(B_P, n))) break;
                tc_fence_after();
                product_ts(tmem + T_O2, tmem + T_A, v, VW, TCH / 16, false);
                if (!(ok = wait(B_K, n))) break;
                tc_fence_after();
                // a tile of one panel gives its columns twice; the upper lanes are not read
                Tile khi{k.at, KW == 64 ? 0u : PANEL, true}, klo{q.at, KW == 64 ? 0u : PANEL, true};
                product(tmem + T_U, khi, v, VW, TCH / 16, false);
                product(tmem + T_U, klo, v, VW, TCH / 16, true);
                commit(bar(B_U));
                if (n + 1 < N) {
                    const int s = int((n + 1) & 1);
                    // P lies where the next A goes
                    if (!(ok = wait(B_FULL0 + s, (n + 1) >> 1) && wait(B_U, n))) break;
                    tc_fence_after();
                    tiles(n + 1, q, k, v);
                    product(tmem + T_A, q, k, TCH, kd, false);
                    commit(bar(B_A));
                }
            }
            int quiet = 0;
            commit(bar(B_END));
            mbar_wait(bar(B_END), 0, &quiet, status);
        }
        __syncwarp();
    } else {
        const int wq = warp & 3, g = warp >> 2, i = wq * 32 + lane, c0 = g * VH;
        const uint32_t lanes = tmem + (uint32_t(wq * 32) << 16);
        float S[VH];
        const int64_t dd = int64_t(a.Dk) * a.Dv;
        load_part<VH>(S, nseg > 1 ? a.S + int64_t(blockIdx.x) * dd : a.s0 ? a.s0 + seg.bh * dd : nullptr, i, c0, a);
        auto put_state = [&]() {
            if (i < KW) {
#pragma unroll
                for (int u = 0; u < VH; u += 32) put32(S_AT, SPANEL, i, c0 + u, reinterpret_cast<const float(&)[32]>(S[u]));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_S));
        };
        put_state();
        for (int64_t n = 0; n < N; ++n) {
            const int s = int(n & 1);
            const uint32_t Q = base + s * STAGE, K = Q + TILE_K, V = K + TILE_K;
            const ChunkDecay &d = dec[s];
            bool ok = all_ok(wait(B_DEC0 + s, n >> 1) && wait(B_A, n));
            // P: this thread's row i, columns 16 g .. + 16 of every block of 32
            float A[4][16];
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (c <= wq) ld16(lanes + T_A + 32 * c + 16 * g, A[c]);
                tc_fence_before();
            }
            // P goes where A was: the warp that shares these lanes has read its columns
            asm volatile("bar.sync %0, 64;" ::"r"(2 + wq) : "memory");
            if (ok) {
                tc_fence_after();
                const float xi = d.x[i];
                const int ri = d.r[i];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[8];
                    const int j0 = 32 * c + 16 * g;
                    if (c < wq) {
                        const float f = ri == d.re[c]
                                            ? fast_exp2((d.Ehi[wq] - d.Ehi[c]) + (d.Elo[wq] - d.Elo[c]) + xi) : 0.f;
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float w0 = d.wb[j0 + e] * f, w1 = d.wb[j0 + e + 1] * f;
                            p[e / 2] = pack(w0 == 0.f ? 0.f : A[c][e] * w0, w1 == 0.f ? 0.f : A[c][e + 1] * w1);
                        }
                    } else if (c == wq) {
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            float y[2];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int j = j0 + e + h;
                                y[h] = j <= i && ri == d.r[j] ? A[c][e + h] * fast_exp2(xi - d.x[j]) : 0.f;
                            }
                            p[e / 2] = pack(y[0], y[1]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) p[e] = 0u;
                    }
                    st8(lanes + T_A + 16 * c + 8 * g, p);
                }
                st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_P));
            }
            // l K: the first products are done with Q and K, whose tiles take the two parts
            ok = ok && all_ok(wait(B_O1, n));
            if (ok) {
                scale_row(K, Q, PANEL, i, g * (KW / 16), (g + 1) * (KW / 16), d.to_end(i));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_K));
            }
            ok = ok && all_ok(wait(B_U, n));
            if (ok) {
                tc_fence_after();
                const float tot = d.total;
#pragma unroll
                for (int u = 0; u < VH; u += 32) {
                    float x[32];
                    ld32(lanes + T_U + c0 + u, x);
#pragma unroll
                    for (int e = 0; e < 32; ++e) S[u + e] = tot == 0.f ? x[e] : fmaf(tot, S[u + e], x[e]);
                }
                tc_fence_before();
                put_state();
                // outputs, through V's tile
                const float f = d.first(i);
#pragma unroll
                for (int u = 0; u < VH; u += 32) {
                    float x[32], y[32];
                    ld32(lanes + T_O1 + c0 + u, x);
                    ld32(lanes + T_O2 + c0 + u, y);
#pragma unroll
                    for (int e = 0; e < 32; ++e) y[e] = a.scale * (f == 0.f ? y[e] : fmaf(f, x[e], y[e]));
                    put32(V, PANEL, i, c0 + u, y);
                }
                tc_fence_before();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_OFREE));
            }
            if (!bar_red_and(1, CW * 32, ok)) break;
            if (threadIdx.x == 0) {
                for (int p = 0; p < VW / 64; ++p)
                    store4(&m.o, p * 64, int(seg.h), int((seg.n0 + n) * TCH), int(seg.b), V + p * PANEL);
                bulk_commit();
                bulk_wait_read();
                mbar_arrive(bar(B_EMPTY0 + s));
            }
        }
        if (a.s1 && seg.n1 == a.NC) store_part<VH>(S, a.s1 + seg.bh * dd, i, c0, a);
        if (threadIdx.x == 0) bulk_wait_all();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W_MMA) {
        tc_fence_after();
        free512(tmem);
    }
}

// ---------------------------------------------------------------- segment states
// The state that a segment's own tokens leave (zero before it): S[blockIdx.x], and the decay
// over it.  REV: the adjoint state from q and scale go, walked from the last chunk back.
template <int KW, int VW>
constexpr size_t state_smem() {
    return 2 * size_t(KW + VW) * 256 + size_t(KW) * 256 + 2 * sizeof(ChunkDecay) + sizeof(Ctl);
}

template <int KW, int VW, bool REV>
__global__ __launch_bounds__(TC_BLOCK, 1) void k_lin_tc_state(const __grid_constant__ StateMaps m, const LinArgs a, int nseg,
                                                              int cps, unsigned *status) {
    constexpr uint32_t STAGE = (KW + VW) * 256, TILE_K = KW * 256, PANEL = TCH * 128;
    constexpr int VH = VW / 2;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t base = smem_u32(sm), LO = base + 2 * STAGE;
    ChunkDecay *dec = reinterpret_cast<ChunkDecay *>(sm + 2 * STAGE + TILE_K);
    Ctl *ctl = reinterpret_cast<Ctl *>(dec + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Seg seg(a, nseg, cps);
    const int64_t N = seg.n1 - seg.n0;
    auto chunk = [&](int64_t n) { return REV ? seg.n1 - 1 - n : seg.n0 + n; };
    if (seg.seg == (REV ? 0 : nseg - 1)) return;     // no segment reads what this one leaves

    if (threadIdx.x == 0) {
        for (int i = 0; i < B_COUNT; ++i) mbar_init(smem_u32(&ctl->bar[i]), i == B_K ? CW : 1);
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
                if (n >= 2 && !wait(B_EMPTY0 + s, (n >> 1) - 1)) break;
                const uint32_t at = base + s * STAGE, b = bar(B_FULL0 + s);
                const int t = int(chunk(n) * TCH);
                mbar_arrive_expect_tx(b, STAGE);
                for (int p = 0; p < KW / 64; ++p) load4(at + p * PANEL, &m.x, p * 64, int(seg.hk), t, int(seg.b), b);
                for (int p = 0; p < VW / 64; ++p) load4(at + TILE_K + p * PANEL, &m.y, p * 64, int(seg.h), t, int(seg.b), b);
            }
            int quiet = 0;
            for (int64_t i = n > 2 ? n - 2 : 0; i < n; ++i) mbar_wait(bar(B_FULL0 + int(i & 1)), uint32_t((i >> 1) & 1), &quiet, status);
        }
        __syncwarp();
    } else if (warp == W_DEC) {
        double sum = 0.0;
        int cuts = 0;
        for (int64_t n = 0; n < N; ++n) {
            const int s = int(n & 1);
            if (n >= 2 && !all_ok(wait(B_EMPTY0 + s, (n >> 1) - 1))) break;
            const int64_t t = chunk(n) * TCH;
            sum += dec[s].fill(a.g + (seg.b * a.T + t) * a.H + seg.h, a.H, int(a.T - t < TCH ? a.T - t : TCH));
            __syncwarp();
            cuts += dec[s].n_cut;
            if (lane == 0) mbar_arrive(bar(B_DEC0 + s));
        }
        if (lane == 0) a.tot[blockIdx.x] = cuts ? 0.f : fast_exp2(float(sum));
    } else if (warp == W_MMA) {
        if (lane == 0) {
            for (int64_t n = 0; n < N; ++n) {
                const int s = int(n & 1);
                if (!(wait(B_FULL0 + s, n >> 1) && wait(B_K, n))) break;
                tc_fence_after();
                const uint32_t at = base + s * STAGE, wide = KW == 64 ? 0u : PANEL;
                const Tile y{at + TILE_K, PANEL, true};
                product(tmem, Tile{at, wide, true}, y, VW, TCH / 16, false);
                product(tmem, Tile{LO, wide, true}, y, VW, TCH / 16, true);
                commit(bar(B_U));
            }
            int quiet = 0;
            commit(bar(B_END));
            mbar_wait(bar(B_END), 0, &quiet, status);
        }
        __syncwarp();
    } else {
        const int wq = warp & 3, g = warp >> 2, i = wq * 32 + lane, c0 = g * VH;
        const uint32_t lanes = tmem + (uint32_t(wq * 32) << 16);
        float S[VH];
#pragma unroll
        for (int u = 0; u < VH; ++u) S[u] = 0.f;
        for (int64_t n = 0; n < N; ++n) {
            const int s = int(n & 1);
            const ChunkDecay &d = dec[s];
            bool ok = all_ok(wait(B_FULL0 + s, n >> 1) && wait(B_DEC0 + s, n >> 1));
            if (ok) {
                scale_row(base + s * STAGE, LO, PANEL, i, g * (KW / 16), (g + 1) * (KW / 16),
                          REV ? d.first(i) * a.scale : d.to_end(i));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_K));
            }
            const float tot = d.total;
            ok = ok && all_ok(wait(B_U, n));
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int u = 0; u < VH; u += 32) {
                    float x[32];
                    ld32(lanes + c0 + u, x);
#pragma unroll
                    for (int e = 0; e < 32; ++e) S[u + e] = tot == 0.f ? x[e] : fmaf(tot, S[u + e], x[e]);
                }
                tc_fence_before();
            }
            // every warp is done with the stage, its decays and the accumulator
            if (!bar_red_and(1, CW * 32, ok)) break;
            if (threadIdx.x == 0) mbar_arrive(bar(B_EMPTY0 + s));
        }
        float *out = (REV ? a.dS : a.S) + int64_t(blockIdx.x) * a.Dk * a.Dv;
        store_part<VH>(S, out, i, c0, a);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W_MMA) {
        tc_fence_after();
        free512(tmem);
    }
}

#define LIN_CUDA(x)                           \
    do {                                      \
        cudaError_t e_ = (x);                 \
        if (e_ != cudaSuccess) return e_;     \
    } while (0)

template <int KW, int VW, bool REV>
cudaError_t run_states(const LinArgs &a, const LinSplit &sp, unsigned *status, cudaStream_t st) {
    StateMaps m;
    const bool ok = REV ? map_tokens(&m.x, a.q, a.Dk, a.Hk, a.T, a.B, a.ldq) && map_tokens(&m.y, a.go, a.Dv, a.H, a.T, a.B, a.ldo)
                        : map_tokens(&m.x, a.k, a.Dk, a.Hk, a.T, a.B, a.ldk) && map_tokens(&m.y, a.v, a.Dv, a.H, a.T, a.B, a.ldv);
    if (!ok) return cudaErrorInvalidValue;
    constexpr size_t smem = state_smem<KW, VW>();
    LIN_CUDA(cudaFuncSetAttribute(k_lin_tc_state<KW, VW, REV>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)));
    ProfScope ps(K_LIN_STATE, st);
    k_lin_tc_state<KW, VW, REV><<<unsigned(a.B * a.H * sp.nseg), TC_BLOCK, smem, st>>>(m, a, sp.nseg, sp.cps, status);
    return cudaGetLastError();
}

template <int KW, int VW>
cudaError_t run_fwd(const LinArgs &a, const LinSplit &sp, unsigned *status, cudaStream_t st) {
    static_assert(fwd_smem<128, 128>() <= 232448 && state_smem<128, 128>() <= 232448, "shared memory of an SM");
    FwdMaps m;
    if (!map_tokens(&m.q, a.q, a.Dk, a.Hk, a.T, a.B, a.ldq) || !map_tokens(&m.k, a.k, a.Dk, a.Hk, a.T, a.B, a.ldk) ||
        !map_tokens(&m.v, a.v, a.Dv, a.H, a.T, a.B, a.ldv) || !map_tokens(&m.o, a.o, a.Dv, a.H, a.T, a.B, a.ldo))
        return cudaErrorInvalidValue;
    if (sp.nseg > 1) {
        LIN_CUDA((run_states<KW, VW, false>(a, sp, status, st)));
        LinArgs b = a;
        b.s1 = nullptr;                 // the last segment writes it
        LIN_CUDA(launch_lin_scan(b, sp.nseg, false, st));
    }
    constexpr size_t smem = fwd_smem<KW, VW>();
    LIN_CUDA(cudaFuncSetAttribute(k_lin_tc_fwd<KW, VW>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)));
    ProfScope ps(K_LIN_OUT, st);
    k_lin_tc_fwd<KW, VW><<<unsigned(a.B * a.H * sp.nseg), TC_BLOCK, smem, st>>>(m, a, sp.nseg, sp.cps, status);
    return cudaGetLastError();
}

}  // namespace

LinSplit lin_split(const LinArgs &a) {
    const int64_t heads = a.B * a.H, NC = cdiv(a.T, TCH);
    LinSplit s{1, int(NC)};
    // One block an SM: split the tokens when that fills SMs that would stay idle; a segment is at
    // least four chunks, below which its start costs more than it saves.
    if (heads < 152 && NC >= 8) {
        int64_t n = std::min<int64_t>(152 / heads, NC / 4);
        if (n > 1) {
            s.cps = int(cdiv(NC, n));
            s.nseg = int(cdiv(NC, s.cps));
        }
    }
    return s;
}

cudaError_t launch_lin_tc_fwd(const LinArgs &args, unsigned *status, cudaStream_t st) {
    LinArgs a = args;
    a.NC = cdiv(a.T, TCH);
    const LinSplit sp = lin_split(a);
    if (a.Dk <= 64) return a.Dv <= 64 ? run_fwd<64, 64>(a, sp, status, st) : run_fwd<64, 128>(a, sp, status, st);
    return a.Dv <= 64 ? run_fwd<128, 64>(a, sp, status, st) : run_fwd<128, 128>(a, sp, status, st);
}

}  // namespace adj
