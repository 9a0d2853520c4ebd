// adj_sample.cu -- sampling a token with temperature, min-p, top-k and top-p from given random
// numbers.  include/adj.h defines it.
//
// Weights are whole numbers, w = round(2^40 e^((x - m) / temperature)): their sums do not depend on the
// order, so any number of threads and blocks gives the same token.  They are formed with 42 bits from
// pairs of fp32 (the fp64 pipe would take the whole time): (x - m) log2 e / temperature as a pair t + e,
// 2^-t from a table of 256 steps and the rest, below 2^-9, from its series.
//
// The kept tokens are a prefix of the order by x, so a limit is a key (the order of the fp32 values as
// unsigned integers) and a number of tokens that equal it.  Top-k and top-p are found without sorting:
// counts and weights over 2048 bins of distance from the maximum say in which bin a limit lies; the keys
// of that bin are cut into 2048 parts again until one key is left, at most three times (one distinct
// value in a bin, as often with bf16, ends it at once).  The token is then found by index: sums of the
// kept weights of every warp's part, of every thread's share of the part that holds it, and along
// that share.
//
// One cluster of 1 to 8 blocks a row; the first pass over the logits comes from HBM and the others
// find them in L2.
#include <algorithm>

#include "adj_profile.cuh"
#include "adj_row.cuh"
#include "adj_seq.cuh"

namespace adj {
namespace {

constexpr int ST = 512;                 // threads of a block
constexpr int SW = ST / 32;
constexpr int BINS = 2048;
constexpr uint64_t ONE = uint64_t(1) << 40;
constexpr float DEAD = 41.5f;           // 2^-41.5 is less than half a unit
constexpr float PARTS = 48.f;           // bins a power of two: DEAD of them fit

// 2^(-i / 256): as a whole number of 2^-42, and as a pair of fp32
struct alignas(16) Step {
    unsigned long long fixed;
    float hi, lo;
};
struct StepTable {
    Step s[256];
};
constexpr StepTable make_steps() {
    StepTable t{};
    const double root = 0.99729605608547012625;         // 2^(-1/256)
    double v = 1.0;
    for (int i = 0; i < 256; ++i) {
        t.s[i].fixed = static_cast<unsigned long long>(v * 4398046511104.0 + 0.5);
        t.s[i].hi = static_cast<float>(v);
        t.s[i].lo = static_cast<float>(v - static_cast<double>(t.s[i].hi));
        v *= root;
    }
    return t;
}
__device__ const StepTable g_steps = make_steps();

// A row's weights
struct Weigh {
    float m, hi, lo;                    // the largest logit; log2 e / temperature as a pair
    bool greedy;
    const Step *steps;

    // a part of the distances from the largest: never falls as x does; -1: too far
    __device__ __forceinline__ int bin(float x) const {
        const float t = (m - x) * hi;
        return x == m ? 0 : t < DEAD ? int(t * PARTS) : -1;
    }
    __device__ __forceinline__ uint64_t operator()(float x) const {
        if (x == m) return ONE;
        const float d = m - x, t = d * hi;
        if (greedy || !(t < DEAD)) return 0;            // NaN: minus infinity at an infinite temperature
        const float b = d - m, dl = (m - (d - b)) - (x + b);
        const float e = fmaf(d, hi, -t) + fmaf(d, lo, dl * hi);
        const float MAGIC = 12582912.f;                 // 1.5 2^23: rounds to whole numbers
        const float kf = fmaf(t, 256.f, MAGIC);
        const int k = __float_as_int(kf) - __float_as_int(MAGIC);
        const float r = fmaf(kf - MAGIC, -1.f / 256.f, t);      // exact
        constexpr float L = 0.693147182464599609375f, LL = -1.904654323148236017e-9f;
        const float ph = -r * L, pl = fmaf(-r, L, -ph);
        const float sq = ph * ph, tail = fmaf(sq, fmaf(ph, fmaf(ph, 1.f / 24.f, 1.f / 6.f), 0.5f), fmaf(-e, L, fmaf(-r, LL, pl)));
        const Step s = steps[k & 255];
        const float q = s.hi * ph, low = fmaf(s.hi, ph, -q) + fmaf(s.lo, ph, s.hi * tail);
        const float qa = fmaf(q, 1048576.f, MAGIC);             // 2^20
        const float rest = fmaf(qa - MAGIC, -1.f / 1048576.f, q) + low;
        const float qb = fmaf(rest, 4398046511104.f, MAGIC);    // 2^42, below 2^22 of it
        const long long whole = (long long)s.fixed + ((long long)(__float_as_int(qa) - __float_as_int(MAGIC)) << 22) +
                                (__float_as_int(qb) - __float_as_int(MAGIC));
        const int n = (k >> 8) + 2;
        return uint64_t(whole + (1ll << (n - 1))) >> n;
    }
};

struct Shared {
    Step steps[256];
    unsigned long long weight[BINS];
    uint32_t count[BINS];
    // what the blocks of a cluster read of one another
    float top;
    uint32_t bad, kmin, kmax;
    unsigned long long part[SW];
    uint32_t ties[SW];
    // scratch of a block
    unsigned long long red64[SW];
    uint32_t red32[SW];
    // a crossing: its bin, what lies before it
    uint32_t bin, before_c, owner, owner_ties;
    unsigned long long before_w, owner_w, total;
};

// Exclusive sums over the block's threads, in their order; totals in every thread.
__device__ void block_scan(Shared &s, uint32_t c, uint64_t w, uint32_t &ec, uint64_t &ew, uint32_t &tc, uint64_t &tw) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t ic = c;
    uint64_t iw = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t x = __shfl_up_sync(~0u, ic, d);
        const uint64_t y = __shfl_up_sync(~0u, iw, d);
        if (lane >= d) {
            ic += x;
            iw += y;
        }
    }
    __syncthreads();
    if (lane == 31) {
        s.red32[warp] = ic;
        s.red64[warp] = iw;
    }
    __syncthreads();
    uint32_t bc = 0;
    uint64_t bw = 0;
    tc = 0;
    tw = 0;
#pragma unroll
    for (int i = 0; i < SW; ++i) {
        if (i < warp) {
            bc += s.red32[i];
            bw += s.red64[i];
        }
        tc += s.red32[i];
        tw += s.red64[i];
    }
    ec = bc + ic - c;
    ew = bw + iw - w;
}

// Four bins of a thread over all blocks, with what lies in the bins before them
struct Level {
    static constexpr int PER = BINS / ST;
    uint32_t c[PER], before_c, all_c;
    uint64_t w[PER], before_w, all_w;
    __device__ void read(Shared &s, int blocks) {
        uint32_t sc = 0;
        uint64_t sw = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int bin = int(threadIdx.x) * PER + i;
            c[i] = s.count[bin];
            w[i] = s.weight[bin];
        }
        if (blocks > 1) {
#pragma unroll
            for (int i = 0; i < PER; ++i) c[i] = 0, w[i] = 0;
            for (int b = 0; b < blocks; ++b)
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int bin = int(threadIdx.x) * PER + i;
                    c[i] += peer(s.count + bin, b);
                    w[i] += peer(s.weight + bin, b);
                }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            sc += c[i];
            sw += w[i];
        }
        block_scan(s, sc, sw, before_c, before_w, all_c, all_w);
    }
};

// A limit being looked for: the first `k` tokens, or those before which less than `mass` lies
struct Goal {
    bool by_count;
    uint32_t k;
    double mass;
    __device__ __forceinline__ bool inside(uint32_t c, uint64_t w) const { return by_count ? c < k : double(w) < mass; }
};

// The last bin whose beginning is inside the goal, given what lies before the whole level.
__device__ void cross(Shared &s, const Level &l, const Goal &g, uint32_t over_c, uint64_t over_w) {
    uint32_t c = over_c + l.before_c;
    uint64_t w = over_w + l.before_w;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < Level::PER; ++i) {
        if (l.c[i] && g.inside(c, w) && !g.inside(c + l.c[i], w + l.w[i])) {
            s.bin = threadIdx.x * Level::PER + i;
            s.before_c = c;
            s.before_w = w;
        }
        c += l.c[i];
        w += l.w[i];
    }
    __syncthreads();
}

// A limit: tokens above `key`, and the first `ties` of those that equal it, hold `weight`
struct Cut {
    uint32_t key, ties;
    uint64_t weight;
};

template <class T>
struct Row {
    static constexpr int N = Vec<T>::N;
    Ragged<T> x;
    int v0, nv;                         // this block's vectors
    __device__ Row(const SampleArgs &a, int64_t row, int blocks, uint32_t rank)
        : x(const_cast<T *>(static_cast<const T *>(a.logits)) + row * a.ld, a.V) {
        const int all = int(x.vectors()), per = (all + blocks - 1) / blocks;
        v0 = int(rank) * per;
        nv = max(0, min(all - v0, per));
    }
    __device__ __forceinline__ void load(int i, float (&v)[N]) const { x.load(v0 + i, v, -INFINITY); }
    __device__ __forceinline__ int64_t index(int i, int e) const { return int64_t(v0 + i) * N - x.shift + e; }
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        for (int i = threadIdx.x; i < nv; i += ST) {
            float v[N];
            load(i, v);
#pragma unroll
            for (int e = 0; e < N; ++e) f(v[e]);
        }
    }
};

__device__ __forceinline__ void clear(Shared &s) {
    for (int i = threadIdx.x; i < BINS; i += ST) {
        s.count[i] = 0;
        s.weight[i] = 0;
    }
}

// The limit in bin s.bin of the distances: the keys there, cut again until one is left.
template <class T>
__device__ Cut narrow(Shared &s, const Row<T> &row, const Weigh &weigh, uint64_t least, const Goal &g, int blocks) {
    const int bin = int(s.bin);
    uint32_t over_c = s.before_c, lo = ~0u, hi = 0;
    uint64_t over_w = s.before_w;
    meet(blocks);                                                   // everyone has read what a call before left
    row.each([&](float x) {
        if (weigh.bin(x) != bin || weigh(x) < least) return;
        const uint32_t k = order_key(x);
        lo = min(lo, k);
        hi = max(hi, k);
    });
    lo = __reduce_min_sync(~0u, lo);
    hi = __reduce_max_sync(~0u, hi);
    if (threadIdx.x == 0) {
        s.kmin = ~0u;
        s.kmax = 0;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        atomicMin(&s.kmin, lo);
        atomicMax(&s.kmax, hi);
    }
    meet(blocks);
    lo = s.kmin;
    hi = s.kmax;
    for (int b = 0; blocks > 1 && b < blocks; ++b) {
        lo = min(lo, peer(&s.kmin, b));
        hi = max(hi, peer(&s.kmax, b));
    }
    while (lo < hi) {
        const int shift = max(0, 21 - __clz(hi - lo));              // the range in at most 2048 parts
        meet(blocks);                                               // everyone has read the bins before
        clear(s);
        __syncthreads();
        row.each([&](float x) {
            const uint32_t k = order_key(x);
            if (k < lo || k > hi) return;
            const uint64_t w = weigh(x);
            if (w < least) return;
            atomicAdd(&s.count[(hi - k) >> shift], 1u);
            atomicAdd(&s.weight[(hi - k) >> shift], (unsigned long long)w);
        });
        meet(blocks);
        Level l;
        l.read(s, blocks);
        cross(s, l, g, over_c, over_w);
        over_c = s.before_c;
        over_w = s.before_w;
        hi -= s.bin << shift;
        lo = max(lo, hi - ((1u << shift) - 1));
    }
    Cut c{hi, 0, over_w};
    const uint64_t w = weigh(key_value(hi));
    if (w == 0) return c;                                           // not reached: a bin that is crossed holds a token
    if (g.by_count) {
        c.ties = g.k - over_c;
    } else {
        uint64_t n = uint64_t(fmax((g.mass - double(over_w)) / double(w), 1.0));
        while (double(over_w + n * w) < g.mass) ++n;
        while (n > 1 && !(double(over_w + (n - 1) * w) < g.mass)) --n;
        c.ties = uint32_t(n);
    }
    c.weight += c.ties * w;
    return c;
}

template <class T>
__global__ __launch_bounds__(ST, 2) void k_sample(const SampleArgs a, int blocks) {
    constexpr int N = Vec<T>::N;
    extern __shared__ __align__(16) char raw[];
    Shared &s = *reinterpret_cast<Shared *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = blocks > 1 ? rank_in_cluster() : 0u;
    const int64_t n = int64_t(blockIdx.x) / blocks;
    const Row<T> row(a, n, blocks, rank);

    const float temperature = a.temperature ? a.temperature[n] : 1.f;
    const float top_p = a.top_p ? a.top_p[n] : 1.f, min_p = a.min_p ? a.min_p[n] : 0.f;
    const int32_t top_k = a.top_k ? a.top_k[n] : 0;
    float top = -INFINITY;
    bool bad = !(temperature >= 0.f) || top_p != top_p || min_p != min_p;
    if (tid < 256) s.steps[tid] = g_steps.s[tid];
    clear(s);
    if (tid == 0) s.bad = 0;
    row.each([&](float x) {
        bad |= !(x < INFINITY);                                     // NaN or +inf
        top = fmaxf(top, x);
    });
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    __syncthreads();
    if (lane == 0) s.red32[warp] = __float_as_uint(top);
    if (bad) s.bad = 1;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SW; ++i) top = fmaxf(top, __uint_as_float(s.red32[i]));
    if (tid == 0) s.top = top;
    meet(blocks);
    bad = s.bad;
    for (int b = 0; blocks > 1 && b < blocks; ++b) {
        top = fmaxf(top, peer(&s.top, b));
        bad |= peer(&s.bad, b) != 0;
    }
    if (bad || top == -INFINITY) {                                  // every block of the row alike
        if (rank == 0 && tid == 0) {
            a.token[n] = -1;
            if (a.logp) a.logp[n] = bad ? NAN : -INFINITY;
        }
        meet(blocks);
        return;
    }
    Weigh weigh;
    weigh.m = top;
    weigh.greedy = temperature == 0.f;
    weigh.steps = s.steps;
    {
        const double c = 1.4426950408889634074 / double(temperature);
        weigh.hi = float(c);
        weigh.lo = float(c - double(weigh.hi));
    }
    const uint64_t least = !(min_p > 0.f) ? 1 : min_p >= 1.f ? ONE : max(uint64_t(1), uint64_t(ceil(double(min_p) * double(ONE))));
    Cut cut{0, 0, 0};                                               // everything
    const bool by_k = top_k > 0 && top_k < a.V, by_p = top_p < 1.f;
    if (weigh.greedy || (by_k && top_k == 1)) {
        cut = Cut{order_key(top), 1, ONE};
    } else if (by_k || by_p) {
        row.each([&](float x) {
            const uint64_t w = weigh(x);
            if (w < least) return;
            const int bin = weigh.bin(x);
            atomicAdd(&s.count[bin], 1u);
            atomicAdd(&s.weight[bin], (unsigned long long)w);
        });
        meet(blocks);
        Level l;
        l.read(s, blocks);
        uint64_t Z = l.all_w;
        if (by_k && uint32_t(top_k) < l.all_c) {
            const Goal g{true, uint32_t(top_k), 0.0};
            cross(s, l, g, 0, 0);
            cut = narrow(s, row, weigh, least, g, blocks);
            Z = cut.weight;
        }
        if (by_p) {
            // one token at least: the first begins below one unit
            const Goal g{false, 0, fmax(double(top_p) * double(Z), 1.0)};
            cross(s, l, g, 0, 0);
            cut = narrow(s, row, weigh, least, g, blocks);
        }
    }

    // The token, by index: this warp's vectors, their kept weight and the number that equal the limit
    const uint64_t tie_w = cut.ties ? weigh(key_value(cut.key)) : 0;
    const int per = (row.nv + SW - 1) / SW, i0 = min(row.nv, warp * per), i1 = min(row.nv, i0 + per);
    auto add = [&](int i, uint64_t &w, uint32_t &t) {
        float v[N];
        row.load(i, v);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const uint32_t k = order_key(v[e]);
            if (k > cut.key) {
                const uint64_t x = weigh(v[e]);
                w += x < least ? 0 : x;
            } else {
                t += k == cut.key;
            }
        }
    };
    uint64_t w = 0;
    uint32_t t = 0;
    for (int i = i0 + lane; i < i1; i += 32) add(i, w, t);
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        w += __shfl_xor_sync(~0u, w, d);
        t += __shfl_xor_sync(~0u, t, d);
    }
    if (lane == 0) {
        s.part[warp] = w;
        s.ties[warp] = t;
    }
    meet(blocks);
    auto kept = [&](uint32_t before, uint32_t t) { return before >= cut.ties ? 0u : min(t, cut.ties - before); };
    {
        // over the warps of all blocks: thread i takes warp i
        const int all = SW * blocks;
        uint64_t pw = 0;
        uint32_t pt = 0, bt, at, u32;
        uint64_t bw, aw;
        if (tid < all) {
            pw = blocks > 1 ? peer(s.part + tid % SW, tid / SW) : s.part[tid];
            pt = blocks > 1 ? peer(s.ties + tid % SW, tid / SW) : s.ties[tid];
        }
        block_scan(s, pt, 0, bt, bw, at, aw);
        const uint64_t mine = pw + kept(bt, pt) * tie_w;
        block_scan(s, 0, mine, u32, bw, at, aw);
        const float u = a.u[n];
        const double goal = double(u > 0.f ? fminf(u, 0.99999994f) : 0.f) * double(aw);
        if (mine && !(double(bw) > goal) && double(bw + mine) > goal) {
            s.owner = uint32_t(tid);
            s.owner_w = bw;
            s.owner_ties = bt;
            s.total = aw;
        }
        __syncthreads();
    }
    meet(blocks);                                                   // all have read what they need of the others
    if (s.owner / SW != rank) return;
    {
        const float u = a.u[n];
        const double goal = double(u > 0.f ? fminf(u, 0.99999994f) : 0.f) * double(s.total);
        const int first = min(row.nv, int(s.owner % SW) * per), last = min(row.nv, first + per);
        const int share = (last - first + ST - 1) / ST, j0 = min(last, first + tid * share), j1 = min(last, j0 + share);
        w = 0;
        t = 0;
        for (int i = j0; i < j1; ++i) add(i, w, t);
        uint32_t bt, at, u32;
        uint64_t bw, aw;
        block_scan(s, t, 0, bt, bw, at, aw);
        bt += s.owner_ties;
        const uint64_t mine = w + kept(bt, t) * tie_w;
        block_scan(s, 0, mine, u32, bw, at, aw);
        bw += s.owner_w;
        if (mine && !(double(bw) > goal) && double(bw + mine) > goal) {
            // along this thread's share; the last kept token where rounding passes over the goal
            int64_t token = -1;
            float value = 0.f;
            for (int i = j0; i < j1; ++i) {
                float v[N];
                row.load(i, v);
                for (int e = 0; e < N; ++e) {
                    const uint32_t k = order_key(v[e]);
                    uint64_t x = 0;
                    if (k > cut.key) {
                        x = weigh(v[e]);
                        x = x < least ? 0 : x;
                    } else if (k == cut.key) {
                        x = bt < cut.ties ? tie_w : 0;
                        ++bt;
                    }
                    if (x == 0) continue;
                    bw += x;
                    token = row.index(i, e);
                    value = v[e];
                    if (double(bw) > goal) {
                        i = j1;
                        break;
                    }
                }
            }
            a.token[n] = token;
            if (a.logp) {
                const float far = value == top ? 0.f : (value - top) / temperature;
                a.logp[n] = far - logf(float(double(s.total) / double(ONE)));
            }
        }
    }
}

template <class T>
cudaError_t launch(const SampleArgs &a, cudaStream_t st) {
    // the blocks of a row: as many as still leave every block 4096 values, while rows alone do not fill the SMs
    int blocks = 1;
    while (blocks < 8 && a.N * blocks * 2 <= 152 * 2 && a.V / (blocks * 2) >= 4096) blocks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.N * blocks));
    cfg.blockDim = dim3(ST);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = unsigned(blocks);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = blocks > 1 ? 1 : 0;
    ProfScope p(K_SAMPLE, st);
    return cudaLaunchKernelEx(&cfg, k_sample<T>, a, blocks);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, bool bf16, cudaStream_t st) {
    return bf16 ? launch<__nv_bfloat16>(a, st) : launch<float>(a, st);
}

}  // namespace adj
