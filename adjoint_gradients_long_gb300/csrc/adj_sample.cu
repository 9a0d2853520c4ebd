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
// counts or weights over bins in falling order say in which bin a limit lies.  bf16 has a bin for each of its
// values, nearly, and is done.  fp32 has 24 bins to a power of two of the distance from the maximum: one
// value alone there is the limit; up to 512 tokens are compared with one another; the keys of more are
// cut into 1024 parts again until one is left, three times at most.  Top-k goes first and counts only, so
// that weights are formed for what it keeps.
// The token is then found by index: sums of the kept weights of every warp's part, of every thread's
// share of the part that holds it, and along that share.
//
// One cluster of 1 to 8 blocks a row, each with its part of the row in shared memory: the logits are
// read once, and every later pass finds them there.
//
// Measured: one row of 32000 bf16 with top-k and top-p 20 us in four blocks, 24 in one, which has no meetings (four
// of the cluster there): passes over the row and the bins, each behind barriers of its block; 64 rows of 131072
// bf16 with top-p 40 us; 152 rows of 50001 fp32 with top-p 63 us, bound by the instructions of the weights
// (55 a token, formed for the bins and again for the draw), without a limit 30 us.
#include <algorithm>

#include "adj_lin.cuh"
#include "adj_profile.cuh"
#include "adj_row.cuh"
#include "adj_seq.cuh"

namespace adj {
namespace {

constexpr int MOST_WARPS = 32;
constexpr int BINS = 1024;
constexpr int LIST = 512;               // tokens of a bin that are compared one by one
constexpr float DEAD = 41.5f;           // 2^-41.5 is less than half a unit
constexpr float PARTS = 24.f;           // bins a power of two: DEAD of them fit

// 2^(-(i + 1) / 256), from 1/2 to below 1, as pairs of fp32
struct StepTable {
    float2 s[256];
};
constexpr StepTable make_steps() {
    StepTable t{};
    const double root = 0.99729605608547012625;         // 2^(-1/256)
    double v = 1.0;
    for (int i = 0; i < 256; ++i) {
        v *= root;
        t.s[i].x = static_cast<float>(v);
        t.s[i].y = static_cast<float>(v - static_cast<double>(t.s[i].x));
    }
    t.s[255].x = 0.5f;
    t.s[255].y = 0.f;
    return t;
}
__device__ const StepTable g_steps = make_steps();

// A row's weights
struct Weigh {
    float m, hi, lo;                    // the largest logit; log2 e / temperature as a pair, finite
    const float2 *steps;
    uint64_t least;                     // the smallest weight that min-p keeps, one unit at least
    float sure, never;                  // distances up to which a weight is above `least`, from which below

    // Without a branch: values at all distances go the same way, and those too far are zero at the end (NaN is
    // too far: minus infinity at an infinite temperature).
    __device__ __forceinline__ uint64_t operator()(float x) const {
        const float d = m - x, t = d * hi;
        const float b = d - m, dl = (m - (d - b)) - (x + b);
        const float e = fmaf(d, hi, -t) + fmaf(d, lo, dl * hi);
        constexpr float MAGIC = 12582912.f;             // 1.5 2^23: rounds to whole numbers, its bits' low 22 are zero
        constexpr uint32_t BITS = 0x4B400000u;
        // t = (256 n + i + 1) / 256 + r, i of 0 to 255 and n from -1 on: the bits of kf end in those of 256 n + i
        const float kf = fmaf(t, 256.f, MAGIC - 1.f);
        const uint32_t kb = __float_as_uint(kf);
        const float r = fmaf(kf - (MAGIC - 1.f), -1.f / 256.f, t);      // exact
        constexpr float L = 0.693147182464599609375f, LL = -1.904654323148236017e-9f;
        const float ph = -r * L, pl = fmaf(-r, L, -ph);
        // 2^-(r + e) - 1 = y + y^2 / 2 + y^3 / 6, y = ph + rest (the fourth power is below 2^-42)
        const float rest = fmaf(-e, L, fmaf(-r, LL, pl)), tail = fmaf(ph, fmaf(ph, fmaf(ph, 1.f / 6.f, 0.5f), rest), rest);
        const float2 s = steps[kb & 255];
        const float q = s.x * ph, low = fmaf(s.x, ph, -q) + fmaf(s.y, ph, fmaf(s.x, tail, s.y));
        // s.x + q + low in units of 2^-42: s.x is 24 bits of 2^-24, the others go in units of 2^-20, and what that
        // leaves, below 2^21 units, by itself
        const float sum = q + low, lost = low - (sum - q);
        const float qa = fmaf(sum, 1048576.f, MAGIC);
        const float qb = fmaf(fmaf(qa - MAGIC, -1.f / 1048576.f, sum) + lost, 4398046511104.f, MAGIC);
        const uint32_t upper = ((__float_as_uint(s.x) & 0x7FFFFFu) | 0x800000u) + (__float_as_uint(qa) << 4) - (BITS << 4) -
                               (BITS >> 18);
        uint64_t whole = uint64_t(upper) * (1u << 18) + __float_as_uint(qb);
        // 2^-n of it in units of 2^-40, to the nearest
        whole >>= (kb >> 8) + 1 & 63;
        const uint64_t w = (whole + 1) >> 1;
        return t < DEAD ? w : 0;
    }
    // A part of the distances from the largest: never falls as x does; -1: not kept by min-p, or too far.  The weight
    // itself is looked at on the border alone, out of line: inlined, it would be formed for every value.
    __device__ __forceinline__ int bin(float x) const {
        const float t = (m - x) * hi;
        if (!(t < never) || (t > sure && far_weight(m, hi, lo, steps, x) < least)) return -1;
        return int(t * PARTS);
    }
    __device__ __noinline__ static uint64_t far_weight(float m, float hi, float lo, const float2 *steps, float x) {
        return Weigh{m, hi, lo, steps, 1, 0.f, 0.f}(x);
    }
    __device__ __forceinline__ uint64_t kept(float x) const {
        const uint64_t w = (*this)(x);
        return w < least ? 0 : w;
    }
};

// bf16 has few values, so a row repeats them: those of 2^-8 to 2^7 and their negatives have a bin each, in
// falling order, with smaller and larger ones in three bins that several values share.  Counts are
// then all that a pass has to add up, and a weight is formed once a value, not once a token.
constexpr int KEY_LOW = (119 << 7) - 1, KEY_SPAN = 15 * 128 + 1;    // 0: below; 1..: a value each; KEY_SPAN: above
constexpr int KEYS = 2 * KEY_SPAN + 1;
__device__ __forceinline__ int key_bin(float x) {
    const int bits = __float_as_int(x) >> 16, q = min(max(bits & 0x7FFF, KEY_LOW), KEY_LOW + KEY_SPAN) - KEY_LOW;
    return bits < 0 ? KEY_SPAN + q : KEY_SPAN - q;
}
__device__ __forceinline__ bool one_value(int bin) { return bin != 0 && bin != KEY_SPAN && bin != KEYS - 1; }
__device__ __forceinline__ float bin_value(int bin) {
    const int q = bin > KEY_SPAN ? bin - KEY_SPAN : KEY_SPAN - bin;
    return __int_as_float((q + KEY_LOW) << 16 | (bin > KEY_SPAN ? int(0x80000000u) : 0));
}
template <class T>
constexpr bool KEYED = sizeof(T) == 2;

template <class T>
struct KeyTable {};
template <>
struct KeyTable<__nv_bfloat16> {
    unsigned long long weight[KEYS + 1];                // kept weight of a bin of one value
    uint32_t tokens[KEYS + 1], shared_low[3], shared_high[3];
};

struct Shared {
    float2 steps[256];
    uint32_t count[BINS], low[BINS], high[BINS];        // tokens of a bin; the halves of their weights' sum
    // what the blocks of a cluster read of one another
    float top;
    uint32_t bad, kmin, kmax, listed, list[LIST];
    unsigned long long part[MOST_WARPS];
    uint32_t ties[MOST_WARPS];
    // scratch of a block
    unsigned long long red64[MOST_WARPS], list_w[LIST];
    uint32_t red32[MOST_WARPS], all_list[LIST];
    // a crossing: its bin, what it holds and what lies before it
    uint32_t bin, before_c, owner, owner_ties, limit;
    unsigned long long before_w, owner_w, total, mass;
};

// A 64-bit sum in two native 32-bit additions (64 bits in shared memory are a loop of compare and
// exchange, which tokens of one bin hold up); few weights reach 2^32, so the second is rare.
__device__ __forceinline__ void add_weight(uint32_t *low, uint32_t *high, uint64_t w) {
    const uint32_t lo = uint32_t(w), old = atomicAdd(low, lo);
    const uint32_t hi = uint32_t(w >> 32) + (old + lo < old ? 1u : 0u);
    if (hi) atomicAdd(high, hi);
}

// Exclusive sums over the block's threads, in their order; totals in every thread.
template <int ST>
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
    // every warp sums up the warps' totals by itself
    const bool there = lane < ST / 32;
    uint32_t wc = there ? s.red32[lane] : 0;
    uint64_t ww = there ? s.red64[lane] : 0;
#pragma unroll
    for (int d = 1; d < ST / 32; d <<= 1) {
        const uint32_t x = __shfl_up_sync(~0u, wc, d);
        const uint64_t y = __shfl_up_sync(~0u, ww, d);
        if (lane >= d) {
            wc += x;
            ww += y;
        }
    }
    tc = __shfl_sync(~0u, wc, ST / 32 - 1);
    tw = __shfl_sync(~0u, ww, ST / 32 - 1);
    const uint32_t bc = warp ? __shfl_sync(~0u, wc, warp - 1 & 31) : 0;
    const uint64_t bw = warp ? __shfl_sync(~0u, ww, warp - 1 & 31) : 0;
    ec = bc + ic - c;
    ew = bw + iw - w;
}

// A thread's bins over all blocks, with what lies in the bins before them
template <int ST>
struct Level {
    static constexpr int PER = BINS / ST;
    uint32_t c[PER], before_c, all_c;
    uint64_t w[PER], before_w, all_w;
    __device__ void read(Shared &s, int blocks) {
        uint32_t sc = 0;
        uint64_t sw = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) c[i] = 0, w[i] = 0;
        // a block's values are on their way together: one at a time, each would wait for the other block
        for (int b = 0; b < blocks; ++b) {
            uint32_t n[PER], lo[PER], hi[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int bin = int(threadIdx.x) * PER + i;
                const bool own = blocks == 1;
                n[i] = own ? s.count[bin] : peer(s.count + bin, b);
                lo[i] = own ? s.low[bin] : peer(s.low + bin, b);
                hi[i] = own ? s.high[bin] : peer(s.high + bin, b);
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                c[i] += n[i];
                w[i] += (uint64_t(hi[i]) << 32) + lo[i];
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            sc += c[i];
            sw += w[i];
        }
        block_scan<ST>(s, sc, sw, before_c, before_w, all_c, all_w);
    }
};

// The same over the bins of bf16 values; forms the weights of those of one value
template <int ST>
struct KeyLevel {
    static constexpr int PER = (KEYS + ST - 1) / ST;
    uint32_t c[PER], before_c, all_c;
    uint64_t w[PER], before_w, all_w;
    __device__ void read(Shared &s, KeyTable<__nv_bfloat16> &k, const Weigh &weigh, int blocks) {
        uint32_t sc = 0;
        uint64_t sw = 0;
        // Over the blocks first, by threads side by side: a thread's own bins lie apart from its neighbours', and
        // the other blocks' memory takes that ill.  The sums stand where the weights go afterwards.
        uint32_t *all = reinterpret_cast<uint32_t *>(k.weight);
        if (blocks > 1) {
            for (int bin = threadIdx.x; bin < KEYS; bin += ST) {
                uint32_t n = 0;
                for (int b = 0; b < blocks; ++b) n += peer(k.tokens + bin, b);
                all[bin] = n;
            }
            __syncthreads();
        } else {
            all = k.tokens;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int bin = int(threadIdx.x) * PER + i;
            c[i] = bin < KEYS ? all[bin] : 0;           // the last threads have fewer bins: nothing there may be crossed
        }
        if (blocks > 1) __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int bin = int(threadIdx.x) * PER + i;
            w[i] = 0;
            if (bin >= KEYS) continue;
            if (one_value(bin)) {
                const uint64_t one = weigh.kept(bin_value(bin));
                k.weight[bin] = one;
                if (one == 0) c[i] = 0;
                w[i] = c[i] * one;
            } else {
                const int at = bin == 0 ? 0 : bin == KEY_SPAN ? 1 : 2;
                for (int b = 0; b < blocks; ++b)
                    w[i] += (uint64_t(blocks > 1 ? peer(k.shared_high + at, b) : k.shared_high[at]) << 32) +
                            (blocks > 1 ? peer(k.shared_low + at, b) : k.shared_low[at]);
            }
            sc += c[i];
            sw += w[i];
        }
        block_scan<ST>(s, sc, sw, before_c, before_w, all_c, all_w);
    }
};

// A limit being looked for: the first `k` tokens, or those before which less than `mass` lies
struct Goal {
    bool by_count;
    uint32_t k;
    uint64_t mass;
    __device__ __forceinline__ bool inside(uint32_t c, uint64_t w) const { return by_count ? c < k : w < mass; }
};

// The last bin whose beginning is inside the goal, given what lies before the whole level.
template <class L>
__device__ void cross(Shared &s, const L &l, const Goal &g, uint32_t over_c, uint64_t over_w) {
    uint32_t c = over_c + l.before_c;
    uint64_t w = over_w + l.before_w;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < L::PER; ++i) {
        if ((g.by_count ? l.c[i] != 0 : l.w[i] != 0) && g.inside(c, w) && !g.inside(c + l.c[i], w + l.w[i])) {
            s.bin = threadIdx.x * L::PER + i;
            s.before_c = c;
            s.before_w = w;
        }
        c += l.c[i];
        w += l.w[i];
    }
    __syncthreads();
}

// A limit: tokens above `x`, and the first `ties` of those that equal it; their weight (where weights were added)
struct Cut {
    float x;
    uint32_t ties;
    uint64_t weight;
    // that of equal tokens, of weight w each, which begin with `c` tokens and weight `over` before them
    __device__ __forceinline__ static Cut among(float x, uint64_t w, const Goal &g, uint32_t c, uint64_t over) {
        // a bin that is crossed holds a token: w > 0
        const uint32_t n = w == 0 ? 0 : g.by_count ? g.k - c : uint32_t((g.mass - over + w - 1) / w);
        return Cut{x, n, over + n * w};
    }
};

// A block's part of a row: 16-byte vectors in shared memory, minus infinity where they reach over the row
template <class T, int ST>
struct Row {
    static constexpr int N = Vec<T>::N;
    uint4 *v;
    int nv;                             // vectors
    int64_t j0;                         // index of the first value
    __device__ Row(const SampleArgs &a, int64_t row, int blocks, uint32_t rank, uint4 *to) : v(to) {
        const Ragged<T> x(const_cast<T *>(static_cast<const T *>(a.logits)) + row * a.ld, a.V);
        const int all = int(x.vectors()), per = (all + blocks - 1) / blocks, v0 = int(rank) * per;
        nv = max(0, min(all - v0, per));
        j0 = int64_t(v0) * N - x.shift;
        const uint4 *from = reinterpret_cast<const uint4 *>(x.p - x.shift) + v0;
        // the first and the last vector of the row may lie partly outside it
        const int w0 = nv > 0 && !x.whole(v0) ? 1 : 0, w1 = nv > w0 && !x.whole(v0 + nv - 1) ? nv - 1 : nv;
        for (int i = w0 + int(threadIdx.x); i < w1; i += ST)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(v + i))),
                         "l"(from + i)
                         : "memory");
        if (threadIdx.x < 2 && (threadIdx.x == 0 ? w0 == 1 : w1 < nv)) {
            const int i = threadIdx.x == 0 ? 0 : nv - 1;
            float f[N];
            x.load(v0 + i, f, -INFINITY);
            v[i] = Vec<T>::pack(f);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    __device__ __forceinline__ int64_t index(int i, int e) const { return j0 + int64_t(i) * N + e; }
    template <class F>
    __device__ __forceinline__ void each_of(int i, int end, int step, F f) const {
        for (; i < end; i += step) {
            float x[N];
            Vec<T>::unpack(v[i], x);
#pragma unroll
            for (int e = 0; e < N; ++e) f(x[e]);
        }
    }
    template <class F>
    __device__ __forceinline__ void each(F f) const { each_of(threadIdx.x, nv, ST, f); }
};

template <int ST>
__device__ __forceinline__ void clear(Shared &s) {
    for (int i = threadIdx.x; i < BINS; i += ST) {
        s.count[i] = s.low[i] = s.high[i] = 0;
    }
}

// The limit in bin s.bin, of the distances or of bf16's shared ones, among tokens of at least `floor`.
template <class T, int ST>
__device__ Cut narrow(Shared &s, const Row<T, ST> &row, const Weigh &weigh, const Goal &g, float floor, int blocks) {
    const int tid = threadIdx.x, bin = int(s.bin);
    const bool weights = KEYED<T> || !g.by_count;
    uint32_t over_c = s.before_c, lo = ~0u, hi = 0;
    uint64_t over_w = s.before_w;
    meet(blocks);                                                   // everyone has read what a call before left
    if (tid == 0) {
        s.kmin = ~0u;
        s.kmax = s.listed = 0;
    }
    __syncthreads();
    row.each([&](float x) {
        if (!(x >= floor) || (KEYED<T> ? key_bin(x) != bin || weigh.kept(x) == 0 : weigh.bin(x) != bin)) return;
        const uint32_t k = order_key(x);
        lo = min(lo, k);
        hi = max(hi, k);
        const uint32_t at = atomicAdd(&s.listed, 1u);
        if (at < LIST) s.list[at] = k;
    });
    lo = __reduce_min_sync(~0u, lo);
    hi = __reduce_max_sync(~0u, hi);
    if ((tid & 31) == 0) {
        atomicMin(&s.kmin, lo);
        atomicMax(&s.kmax, hi);
    }
    meet(blocks);
    lo = s.kmin;
    hi = s.kmax;
    uint32_t total = blocks > 1 ? 0 : s.listed;
    for (int b = 0; blocks > 1 && b < blocks; ++b) {
        lo = min(lo, peer(&s.kmin, b));
        hi = max(hi, peer(&s.kmax, b));
        total += peer(&s.listed, b);
    }
    if (total <= LIST && lo < hi) {
        // every token of the bin with all others: what lies above it; the lowest one inside the goal
        int n = 0;
        for (int b = 0; b < blocks; ++b) {
            const int m = int(blocks > 1 ? peer(&s.listed, b) : s.listed);
            if (tid < m && n + tid < LIST) s.all_list[n + tid] = blocks > 1 ? peer(s.list + tid, b) : s.list[tid];
            n += m;
        }
        n = min(n, LIST);
        if (tid == 0) s.limit = ~0u;
        __syncthreads();
        const uint32_t mine = tid < n ? s.all_list[tid] : 0u;
        if (tid < n) s.list_w[tid] = weights ? weigh(key_value(mine)) : 0;
        __syncthreads();
        uint32_t c = over_c;
        uint64_t w = over_w;
        if (tid < n) {
            for (int i = 0; i < n; ++i)
                if (s.all_list[i] > mine) {
                    ++c;
                    w += s.list_w[i];
                }
            if (g.inside(c, w)) atomicMin(&s.limit, mine);
        }
        __syncthreads();
        if (tid < n && mine == s.limit) {                           // equal tokens write the same
            s.before_c = c;
            s.before_w = w;
        }
        __syncthreads();
        lo = hi = s.limit;
        over_c = s.before_c;
        over_w = s.before_w;
    }
    while (lo < hi) {
        const int shift = max(0, 22 - __clz(hi - lo));              // the range in at most 1024 parts
        meet(blocks);                                               // everyone has read the bins before
        clear<ST>(s);
        __syncthreads();
        row.each([&](float x) {
            const uint32_t k = order_key(x);
            if (k < lo || k > hi) return;
            const uint64_t w = weigh.kept(x);
            if (w == 0) return;
            if (g.by_count) atomicAdd(&s.count[(hi - k) >> shift], 1u);
            if (weights) add_weight(&s.low[(hi - k) >> shift], &s.high[(hi - k) >> shift], w);
        });
        meet(blocks);
        Level<ST> l;
        l.read(s, blocks);
        cross(s, l, g, over_c, over_w);
        over_c = s.before_c;
        over_w = s.before_w;
        hi -= s.bin << shift;
        lo = max(lo, hi - ((1u << shift) - 1));
    }
    const float x = key_value(hi);
    return Cut::among(x, weigh(x), g, over_c, over_w);
}

// bytes of shared memory before the row
template <class T>
constexpr size_t FIXED = sizeof(Shared) + (KEYED<T> ? sizeof(KeyTable<T>) + 15 & ~size_t(15) : 0);

template <class T, int ST>
__global__ __launch_bounds__(ST) void k_sample(const SampleArgs a, int blocks) {
    constexpr int N = Vec<T>::N, SW = ST / 32;
    extern __shared__ __align__(16) char raw[];
    Shared &s = *reinterpret_cast<Shared *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = blocks > 1 ? rank_in_cluster() : 0u;
    const int64_t n = int64_t(blockIdx.x) / blocks;

    const float temperature = a.temperature ? a.temperature[n] : 1.f;
    const float top_p = a.top_p ? a.top_p[n] : 1.f, min_p = a.min_p ? a.min_p[n] : 0.f;
    const int32_t top_k = a.top_k ? a.top_k[n] : 0;
    if (tid < 256) s.steps[tid] = g_steps.s[tid];
    clear<ST>(s);
    if (tid == 0) s.bad = 0;
    KeyTable<T> &keys = *reinterpret_cast<KeyTable<T> *>(raw + sizeof(Shared));     // bf16
    if constexpr (KEYED<T>) {
        for (int i = tid; i < KEYS + 1 + 6; i += ST) keys.tokens[i] = 0;            // the shared sums behind them, too
    }
    const Row<T, ST> row(a, n, blocks, rank, reinterpret_cast<uint4 *>(raw + FIXED<T>));
    __syncthreads();
    float top = -INFINITY;
    bool bad = !(temperature >= 0.f) || top_p != top_p || min_p != min_p;
    row.each([&](float x) {
        bad |= !(x < INFINITY);                                     // NaN or +inf
        top = fmaxf(top, x);
    });
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
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
    weigh.steps = s.steps;
    {
        // log2 e / temperature as a pair: the quotient, and the quotient of what it leaves
        constexpr float H = 1.44269502162933349609375f, L = 1.925963033500011079e-8f;
        weigh.hi = temperature == 0.f ? 3.402823466e38f : fminf(H / temperature, 3.402823466e38f);     // -0 too
        // none for an infinite temperature, nor for one near zero (a difference of logits is far there)
        weigh.lo = weigh.hi == 0.f || weigh.hi > 1e37f ? 0.f : (fmaf(-weigh.hi, temperature, H) + L) / temperature;
    }
    weigh.least = 1;
    weigh.sure = 40.5f;                                             // half a unit is at 41
    weigh.never = DEAD;
    if (min_p > 0.f) {
        const float p = fminf(min_p, 1.f), t = -log2f(p);
        weigh.least = max(uint64_t(1), uint64_t(ceilf(p * 1099511627776.f)));     // 2^40 p: exact
        const float out = weigh.least < 1024 ? 2.f : 0.01f;         // outside log2f's error and the weights' rounding
        weigh.sure = fminf(weigh.sure, t - out);
        weigh.never = fminf(weigh.never, t + out);
    }
    // Everything above what has no weight for certain, rounded away from it: a warp whose values all lie below forms none
    // (152 rows of 50001 fp32 with min-p 0.05: 20 us, against 30)
    Cut cut{__fsub_rd(top, weigh.never * 1.001f / weigh.hi), 0, 0};
    const bool by_k = top_k > 0 && top_k < a.V, by_p = top_p < 1.f;
    if (temperature == 0.f || (by_k && top_k == 1)) {
        cut = Cut{top, 1, 0};
    } else if constexpr (KEYED<T>) {
        if (by_k || by_p) {
            row.each([&](float x) {
                if (!((top - x) * weigh.hi < DEAD)) return;
                const int bin = key_bin(x);
                if (one_value(bin)) {
                    atomicAdd(&keys.tokens[bin], 1u);
                } else if (const uint64_t w = weigh.kept(x)) {
                    const int at = bin == 0 ? 0 : bin == KEY_SPAN ? 1 : 2;
                    atomicAdd(&keys.tokens[bin], 1u);
                    add_weight(&keys.shared_low[at], &keys.shared_high[at], w);
                }
            });
            meet(blocks);
            KeyLevel<ST> l;
            l.read(s, keys, weigh, blocks);
            uint64_t Z = l.all_w;
#pragma unroll 1
            for (int phase = by_k && uint32_t(top_k) < l.all_c ? 0 : 1; phase < (by_p ? 2 : 1); ++phase) {
                Goal g{phase == 0, uint32_t(top_k), 0};
                if (phase == 1) {
                    // one token at least: the first begins below one unit.  One thread alone in 64-bit floating point.
                    if (tid == 0) s.mass = uint64_t(ceil(fmax(double(top_p) * double(Z), 1.0)));
                    __syncthreads();
                    g.mass = s.mass;
                }
                cross(s, l, g, 0, 0);
                const int bin = int(s.bin);
                if (one_value(bin)) cut = Cut::among(bin_value(bin), keys.weight[bin], g, s.before_c, s.before_w);
                else cut = narrow(s, row, weigh, g, -INFINITY, blocks);
                Z = cut.weight;
            }
        } else {
            for (int i = tid; i < KEYS; i += ST) keys.weight[i] = one_value(i) ? weigh.kept(bin_value(i)) : 0;
            __syncthreads();
        }
    } else {
        // Top-k first, then top-p among what is left.  Tokens that equal top-k's limit count in full there,
        // which moves nothing: what top_p asks for lies within the kept ones.
#pragma unroll 1
        for (int phase = by_k ? 0 : 1; phase < (by_p ? 2 : 1); ++phase) {
            const bool mass = phase == 1;
            if (mass && by_k) {
                meet(blocks);                                       // everyone has read the bins
                clear<ST>(s);
                __syncthreads();
            }
            uint32_t equal = 0;                                     // tokens at top-k's limit
            if (tid == 0) s.listed = 0;
            __syncthreads();
            row.each([&](float x) {
                const int bin = x >= cut.x ? weigh.bin(x) : -1;
                if (bin < 0) return;
                equal += x == cut.x;
                if (mass) add_weight(&s.low[bin], &s.high[bin], weigh(x));
                else atomicAdd(&s.count[bin], 1u);
            });
            equal = __reduce_add_sync(~0u, equal);
            if (lane == 0 && equal) atomicAdd(&s.listed, equal);
            meet(blocks);
            Level<ST> l;
            l.read(s, blocks);
            Goal g{!mass, uint32_t(top_k), 0};
            if (mass) {
                // one token at least: the first begins below one unit.  One thread alone in 64-bit floating point.
                if (tid == 0) {
                    uint64_t Z = l.all_w;
                    uint32_t all = blocks > 1 ? 0 : s.listed;
                    for (int b = 0; blocks > 1 && b < blocks; ++b) all += peer(&s.listed, b);
                    if (cut.ties) Z -= uint64_t(all - cut.ties) * weigh(cut.x);
                    s.mass = uint64_t(ceil(fmax(double(top_p) * double(Z), 1.0)));
                }
                __syncthreads();
                g.mass = s.mass;
            } else if (uint32_t(top_k) >= l.all_c) {
                continue;
            }
            cross(s, l, g, 0, 0);
            cut = narrow(s, row, weigh, g, cut.x, blocks);
        }
    }

    // The token, by index: this warp's vectors, their kept weight and the number that equal the limit
    const uint64_t tie_w = cut.ties ? weigh(cut.x) : 0;
    const int per = (row.nv + SW - 1) / SW, i0 = min(row.nv, warp * per), i1 = min(row.nv, i0 + per);
    uint64_t w = 0;
    uint32_t t = 0;
    auto weight_of = [&](float x) -> uint64_t {
        if constexpr (KEYED<T>) {
            const int bin = key_bin(x);
            if (one_value(bin)) return keys.weight[bin];
        }
        return weigh.kept(x);
    };
    auto add = [&](float x) {
        if (x > cut.x) w += weight_of(x);
        else t += x == cut.x;
    };
    row.each_of(i0 + lane, i1, 32, add);
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
        block_scan<ST>(s, pt, 0, bt, bw, at, aw);
        const uint64_t mine = pw + kept(bt, pt) * tie_w;
        block_scan<ST>(s, 0, mine, u32, bw, at, aw);
        if (tid == 0) {
            const float u = a.u[n];
            s.mass = uint64_t(double(u > 0.f ? fminf(u, 0.99999994f) : 0.f) * double(aw));
        }
        __syncthreads();
        if (mine && bw <= s.mass && bw + mine > s.mass) {
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
        const uint64_t goal = s.mass;
        const int first = min(row.nv, int(s.owner % SW) * per), last = min(row.nv, first + per);
        const int share = (last - first + ST - 1) / ST, j0 = min(last, first + tid * share), j1 = min(last, j0 + share);
        w = 0;
        t = 0;
        row.each_of(j0, j1, 1, add);
        uint32_t bt, at, u32;
        uint64_t bw, aw;
        block_scan<ST>(s, t, 0, bt, bw, at, aw);
        bt += s.owner_ties;
        const uint64_t mine = w + kept(bt, t) * tie_w;
        block_scan<ST>(s, 0, mine, u32, bw, at, aw);
        bw += s.owner_w;
        if (mine && bw <= goal && bw + mine > goal) {                // along this thread's share
            int64_t token = -1;
            float value = 0.f;
            for (int i = j0; i < j1; ++i) {
                float v[N];
                Vec<T>::unpack(row.v[i], v);
                for (int e = 0; e < N; ++e) {
                    uint64_t x = 0;
                    if (v[e] > cut.x) {
                        x = weight_of(v[e]);
                    } else if (v[e] == cut.x) {
                        x = bt < cut.ties ? tie_w : 0;
                        ++bt;
                    }
                    if (x == 0) continue;
                    bw += x;
                    token = row.index(i, e);
                    value = v[e];
                    if (bw > goal) {
                        i = j1;
                        break;
                    }
                }
            }
            a.token[n] = token;
            if (a.logp) {
                const float far = value == top ? 0.f : (value - top) / temperature;
                a.logp[n] = far - logf(__ull2float_rn(s.total) * (1.f / 1099511627776.f));
            }
        }
    }
}

template <class T>
constexpr size_t MOST = 232448 - FIXED<T> - 64;                     // for a part of a row
static_assert(ADJ_SAMPLE_MAX_V / 8 * 4 + 32 <= MOST<float> && ADJ_SAMPLE_MAX_V / 8 * 2 + 32 <= MOST<__nv_bfloat16>,
              "a row has to fit eight blocks");

template <class T, int ST>
cudaError_t launch_as(const SampleArgs &a, int blocks, size_t smem, cudaStream_t st) {
    const cudaError_t e = allow_smem<k_sample<T, ST>>(232448);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.N * blocks));
    cfg.blockDim = dim3(ST);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = unsigned(blocks);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = blocks > 1 ? 1 : 0;
    ProfScope p(K_SAMPLE, st);
    return cudaLaunchKernelEx(&cfg, k_sample<T, ST>, a, blocks);
}

template <class T>
cudaError_t launch(const SampleArgs &a, cudaStream_t st) {
    // The fewest blocks whose parts fit; then more, while every block keeps 4096 values and there are SMs for all: a row
    // of 32000 bf16 with top-k and top-p takes 19.6 us in four blocks, 21.2 in two, 23.9 in one.
    auto part = [&](int blocks) { return size_t((a.V * sizeof(T) / 16 + 2 + blocks - 1) / blocks) * 16; };
    int blocks = 1;
    while (blocks < 8 && part(blocks) > MOST<T>) blocks *= 2;
    while (blocks < 8 && a.N * blocks * 2 <= 152 && a.V / (blocks * 2) >= 4096) blocks *= 2;
    const size_t smem = FIXED<T> + part(blocks);
    // a part that leaves no room for a second block beside it gets all the SM's threads
    return smem > 113 * 1024 ? launch_as<T, 1024>(a, blocks, smem, st) : launch_as<T, 512>(a, blocks, smem, st);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, bool bf16, cudaStream_t st) {
    return bf16 ? launch<__nv_bfloat16>(a, st) : launch<float>(a, st);
}

}  // namespace adj
