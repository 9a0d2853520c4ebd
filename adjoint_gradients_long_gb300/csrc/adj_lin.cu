// adj_lin.cu -- linear attention with a decay for each head in plain fp32 arithmetic: the
// chunked forward and backward passes and the single-token step.  include/adj.h defines
// the operators.
//
// Chunked form, chunks of C tokens.  With D_ij the decay from token j to token i >= j of a
// chunk (LinDecay), f_i the decay from before the chunk to i, l_j from j to the chunk's end,
// and S the state that enters the chunk:
//     o_i = scale (sum_{j <= i} D_ij (q_i . k_j) v_j + f_i q_i S)
//     S'  = f_{C-1} S + sum_j l_j k_j v_j^T
// and with w_i = scale go_i and Z the adjoint state (the cotangent of S'):
//     dq_i = sum_{j <= i} D_ij (w_i . v_j) k_j + f_i S w_i
//     dk_j = sum_{i >= j} D_ij (w_i . v_j) q_i + l_j Z v_j
//     dv_j = sum_{i >= j} D_ij (q_i . k_j) w_i + l_j Z^T k_j
//     Z_before = f_{C-1} Z + sum_i f_i q_i w_i^T
// dg_t is the sum of everything whose decay passes through token t: pairs j < t <= i inside
// the chunk with W_ij = D_ij (w_i . v_j)(q_i . k_j), sources j < t that leave the chunk,
// tokens i >= t that read the entering state, and the state that crosses the whole chunk:
//     dg_t = sum_{i >= t > j} W_ij + sum_{j < t} l_j k_j . Z v_j + sum_{i >= t} f_i q_i . S w_i
//            + f_{C-1} <Z, S>.
// The first sum is taken as suffix sums of (row sums - column sums) of W without its
// diagonal; no term is a difference of larger ones across chunks.
//
// Passes: (1) every chunk's own contribution to the state, in parallel; (2) a scan over the
// chunks, element by element of the state; (3) every chunk's outputs, in parallel.
//
// fp32 storage keeps to the fp32 pipe; on the tensor cores three bf16 parts would hold its operands, at
// six products for one (not built).  Measured, 4 x 2000 tokens x 16 heads of 64 and 128: 68 us,
// 35 us and 134 us for the passes (7.4 Gflop; the first version, one block an SM and scalar reads of
// shared memory, took 586 us).  The gradients' last pass, k_lin_grad, still has that form: 806 us for
// all passes of the gradients at the same sizes.
#include <algorithm>

#include "adj_lin.cuh"
#include "adj_profile.cuh"

namespace adj {
namespace {

constexpr int LC = LIN_CHUNK;   // tokens of a chunk
constexpr int LP = 132;         // row pitch of a [*][128] fp32 tile: rows 4 banks apart
constexpr int PP = 68;          // row pitch of a [64][64] tile

__device__ __forceinline__ void ld4(const float *p, float (&v)[4]) {
    const float4 x = __ldg(reinterpret_cast<const float4 *>(p));
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
}
__device__ __forceinline__ void ld4(const __nv_bfloat16 *p, float (&v)[4]) {
    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
    v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xFFFF0000u);
    v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xFFFF0000u);
}

// tile[t * pitch + d] = x[t * ld + d] for t < LC, d < D, rows past len zeros; sixteen threads a row.
// Asynchronous: all of a block's tiles are in flight together, until loaded().
__device__ __forceinline__ void load_tile(float *tile, int pitch, const float *x, int64_t ld, int D, int len) {
#pragma unroll
    for (int t = threadIdx.x >> 4; t < LC; t += 16)
#pragma unroll
        for (int d = (threadIdx.x & 15) << 2; d < 128; d += 64) {
            if (d >= D) break;
            const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(tile + t * pitch + d));
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(x + (t < len ? t * ld + d : 0)),
                         "r"(t < len ? 16 : 0)
                         : "memory");
        }
}
__device__ __forceinline__ void loaded() {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
}
// rows times w[t] * mul (w null: mul alone); a weight of zero drops a row whatever it holds
__device__ __forceinline__ void scale_tile(float *tile, int pitch, int D, float mul, const float *w = nullptr) {
    for (int t = threadIdx.x >> 4; t < LC; t += 16) {
        const float m = w ? w[t] * mul : mul;
        for (int d = (threadIdx.x & 15) << 2; d < D; d += 64) {
            float4 *p = reinterpret_cast<float4 *>(tile + t * pitch + d);
            *p = m == 0.f ? f4(0.f) : f4(m) * *p;
        }
    }
}

// acc[r][c] += sum_k A(ty + 16 r, k) B(k, tx + 16 c) with A at a[row * AR + k * AK] and B at
// b[k * BK + col * BC]; columns past `cols` are left out.
template <int R, int NC, int AR, int AK, int BK, int BC>
__device__ __forceinline__ void mm(float (&acc)[R][NC], const float *a, const float *b, int K, int cols) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    a += ty * AR;
    b += tx * BC;
#pragma unroll 2
    for (int k = 0; k < K; k += 4) {
        float x[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (AK == 1) {
                const float4 f = *reinterpret_cast<const float4 *>(a + r * 16 * AR + k);
                x[r][0] = f.x; x[r][1] = f.y; x[r][2] = f.z; x[r][3] = f.w;
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u) x[r][u] = a[r * 16 * AR + (k + u) * AK];
            }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (16 * c >= cols) break;
            float y[4];
            if (BK == 1) {
                const float4 f = *reinterpret_cast<const float4 *>(b + c * 16 * BC + k);
                y[0] = f.x; y[1] = f.y; y[2] = f.z; y[3] = f.w;
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u) y[u] = b[(k + u) * BK + c * 16 * BC];
            }
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int u = 0; u < 4; ++u) acc[r][c] = fmaf(x[r][u], y[u], acc[r][c]);
        }
    }
}

// Outer-product forms: this thread's rows are 4 ty + q (and + 64), its columns 4 tx + q (and + 64),
// so that 256 FMAs take 16 to 24 shared-memory wavefronts.  `cols`: columns in use.
//   A_K: A(row, k) = a[row * ap + k], else a[k * ap + row];  B(k, col) = b[k * bp + col].
template <int R, bool A_K>
__device__ __forceinline__ void mm_outer(float (&acc)[R][8], const float *a, int ap, const float *b, int bp, int K, int cols) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    a += A_K ? 4 * ty * ap : 4 * ty;
    b += 4 * tx;
    const bool two = cols > 64;
#pragma unroll 2
    for (int k = 0; k < K; k += 4) {
        float x[R][4];          // [row][k]
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (A_K) {
                const float4 f = *reinterpret_cast<const float4 *>(a + ((r & 3) + 64 * (r >> 2)) * ap + k);
                x[r][0] = f.x; x[r][1] = f.y; x[r][2] = f.z; x[r][3] = f.w;
            } else if ((r & 3) == 0) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float4 f = *reinterpret_cast<const float4 *>(a + (k + u) * ap + 16 * r);
                    x[r][u] = f.x; x[r + 1][u] = f.y; x[r + 2][u] = f.z; x[r + 3][u] = f.w;
                }
            }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float4 y = *reinterpret_cast<const float4 *>(b + (k + u) * bp);
            const float4 z = two ? *reinterpret_cast<const float4 *>(b + (k + u) * bp + 64) : f4(0.f);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                acc[r][0] = fmaf(x[r][u], y.x, acc[r][0]);
                acc[r][1] = fmaf(x[r][u], y.y, acc[r][1]);
                acc[r][2] = fmaf(x[r][u], y.z, acc[r][2]);
                acc[r][3] = fmaf(x[r][u], y.w, acc[r][3]);
            }
            if (two)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    acc[r][4] = fmaf(x[r][u], z.x, acc[r][4]);
                    acc[r][5] = fmaf(x[r][u], z.y, acc[r][5]);
                    acc[r][6] = fmaf(x[r][u], z.z, acc[r][6]);
                    acc[r][7] = fmaf(x[r][u], z.w, acc[r][7]);
                }
        }
    }
}

struct At {                     // one chunk of one head
    int64_t b, h, hk, n, t0, seq;
    int len;
    __device__ At(const LinArgs &a) {
        n = blockIdx.x;
        h = blockIdx.y;
        b = blockIdx.z;
        hk = h / (a.H / a.Hk);
        t0 = n * LC;
        len = int(a.T - t0 < LC ? a.T - t0 : LC);
        seq = b * a.T + t0;
    }
    __device__ int64_t state(const LinArgs &a) const { return ((b * a.H + h) * a.NC + n) * a.Dk * a.Dv; }
};
template <class T>
__device__ __forceinline__ const T *row(const void *p, int64_t tok, int64_t ld, int64_t head, int D) {
    return static_cast<const T *>(p) + tok * ld + head * D;
}

// Pitches of tiles D wide: rows an odd multiple of 16 bytes apart, so that 16-byte reads down a
// column of rows meet no bank twice.
__host__ __device__ __forceinline__ int pitch_of(int D) { return D + 4; }

// Pass 1.  REV = false: S[n] = sum_j l_j k_j v_j^T; true: dS[n] = sum_i f_i q_i w_i^T.
template <bool REV>
__global__ __launch_bounds__(256, 3) void k_lin_chunk_state(const LinArgs a) {
    extern __shared__ float sm[];
    const int pk = pitch_of(a.Dk), pv = pitch_of(a.Dv);
    // 64 rows more than a.Dk may be read across A's rows: they lie in B
    float *A = sm, *B = A + LC * pk;
    __shared__ LinDecay<LC> D;
    const At at(a);
    __shared__ float w[LC];
    if (REV) {
        load_tile(A, pk, row<float>(a.q, at.seq, a.ldq, at.hk, a.Dk), a.ldq, a.Dk, at.len);
        load_tile(B, pv, row<float>(a.go, at.seq, a.ldo, at.h, a.Dv), a.ldo, a.Dv, at.len);
    } else {
        load_tile(A, pk, row<float>(a.k, at.seq, a.ldk, at.hk, a.Dk), a.ldk, a.Dk, at.len);
        load_tile(B, pv, row<float>(a.v, at.seq, a.ldv, at.h, a.Dv), a.ldv, a.Dv, at.len);
    }
    if (threadIdx.x < 32) {
        D.fill(a.g + at.seq * a.H + at.h, a.H, at.len);
        __syncwarp();
        for (int t = threadIdx.x; t < LC; t += 32) w[t] = REV ? D.first(t) : D.last(t);
    }
    loaded();
    scale_tile(A, pk, a.Dk, REV ? a.scale : 1.f, w);
    __syncthreads();
    float *S = (REV ? a.dS : a.S) + at.state(a);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    // 64 rows of the state at a time
    for (int d0 = 0; d0 < a.Dk; d0 += 64) {
        float acc[4][8] = {};
        mm_outer<4, false>(acc, A + d0, pk, B, pv, LC, a.Dv);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 8; c += 4) {
                const int d = d0 + 4 * ty + r, e = 4 * tx + 16 * c;
                if (d < a.Dk && e < a.Dv)
                    *reinterpret_cast<float4 *>(S + d * a.Dv + e) = make_float4(acc[r][c], acc[r][c + 1], acc[r][c + 2], acc[r][c + 3]);
            }
    }
    if (threadIdx.x == 0) (REV ? a.dtot : a.tot)[(at.b * a.H + at.h) * a.NC + at.n] = D.total();
}

// Pass 2.  Every chunk's contribution is replaced by the state that enters it (in reverse: by the
// adjoint state that its exit receives); one thread carries four elements through the chunks.
// rev0: the direction of the first half of the grid, the other half (if any) goes the other way.
__global__ __launch_bounds__(128) void k_lin_scan(const LinArgs a, int64_t NC, int64_t half, bool rev0) {
    const bool rev = blockIdx.x < half ? rev0 : !rev0;
    const int64_t block = blockIdx.x < half ? blockIdx.x : blockIdx.x - half;
    const int64_t n4 = int64_t(a.Dk) * a.Dv / 4, blocks = (n4 + 127) / 128, bh = block / blocks;
    const int64_t i = (block - bh * blocks) * 128 + threadIdx.x;
    if (i >= n4) return;
    const float *init = rev ? a.ds1 : a.s0;
    float *fin = rev ? a.ds0 : a.s1;
    float4 c = init ? reinterpret_cast<const float4 *>(init)[bh * n4 + i] : f4(0.f);
    float4 *S = reinterpret_cast<float4 *>(rev ? a.dS : a.S) + bh * NC * n4 + i;
    const float *tot = (rev ? a.dtot : a.tot) + bh * NC;
    constexpr int U = 8;        // loads in flight
    for (int64_t m = 0; m < NC; m += U) {
        float4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (m + u < NC) x[u] = S[(rev ? NC - 1 - m - u : m + u) * n4];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (m + u < NC) {
                const int64_t n = rev ? NC - 1 - m - u : m + u;
                S[n * n4] = c;
                c = tot[n] == 0.f ? x[u] : fma4(f4(tot[n]), c, x[u]);    // a new start drops it whatever it holds
            }
    }
    if (fin) reinterpret_cast<float4 *>(fin)[bh * n4 + i] = c;
}

__device__ __forceinline__ void load_state(float *tile, int pitch, const float *S, int Dk, int Dv) {
    for (int d = threadIdx.x >> 4; d < Dk; d += 16)
#pragma unroll
        for (int e = (threadIdx.x & 15) << 2; e < 128; e += 64) {
            if (e >= Dv) break;
            const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(tile + d * pitch + e));
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(S + int64_t(d) * Dv + e) : "memory");
        }
}

// Pass 3 of the forward pass.
__global__ __launch_bounds__(256, 2) void k_lin_out(const LinArgs a) {
    extern __shared__ float sm[];
    const int pk = pitch_of(a.Dk), pv = pitch_of(a.Dv);
    float *Q = sm, *V = Q + LC * pk, *S = V + LC * pv, *K = S + a.Dk * pv, *P = K;       // P in K's place
    __shared__ LinDecay<LC> D;
    const At at(a);
    load_tile(Q, pk, row<float>(a.q, at.seq, a.ldq, at.hk, a.Dk), a.ldq, a.Dk, at.len);
    load_tile(K, pk, row<float>(a.k, at.seq, a.ldk, at.hk, a.Dk), a.ldk, a.Dk, at.len);
    load_tile(V, pv, row<float>(a.v, at.seq, a.ldv, at.h, a.Dv), a.ldv, a.Dv, at.len);
    load_state(S, pv, a.S + at.state(a), a.Dk, a.Dv);
    if (threadIdx.x < 32) D.fill(a.g + at.seq * a.H + at.h, a.H, at.len);
    loaded();
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    // rows 4 ty + r, columns tx + 16 c
    float p[4][4] = {};
#pragma unroll 2
    for (int k = 0; k < a.Dk; k += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = *reinterpret_cast<const float4 *>(Q + (4 * ty + r) * pk + k);
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] = *reinterpret_cast<const float4 *>(K + (tx + 16 * c) * pk + k);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                p[r][c] = fmaf(x[r].x, y[c].x, fmaf(x[r].y, y[c].y, fmaf(x[r].z, y[c].z, fmaf(x[r].w, y[c].w, p[r][c]))));
    }
    float acc[4][8] = {};
    mm_outer<4, true>(acc, Q, pk, S, pv, a.Dk, a.Dv);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const float f = D.first(4 * ty + r);
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[r][c] = f == 0.f ? 0.f : acc[r][c] * f;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int i = 4 * ty + r, j = tx + 16 * c;
            P[i * PP + j] = j <= i ? p[r][c] * D.pair(i, j) : 0.f;
        }
    __syncthreads();
    // the warp's last row bounds its sums
    mm_outer<4, true>(acc, P, PP, V, pv, 8 * (ty >> 1) + 8, a.Dv);
    float *o = static_cast<float *>(a.o) + at.seq * a.ldo + at.h * a.Dv;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 8; c += 4) {
            const int i = 4 * ty + r, e = 4 * tx + 16 * c;
            if (i < at.len && e < a.Dv)
                st4(o + i * a.ldo + e, make_float4(acc[r][c] * a.scale, acc[r][c + 1] * a.scale, acc[r][c + 2] * a.scale, acc[r][c + 3] * a.scale));
        }
}

// sum over the 16 threads of a row of the thread grid
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int d = 8; d; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
    return x;
}

// dq or dk of one head: to the output, or (shared heads) to the fp32 partials
__device__ __forceinline__ void put_grad(const LinArgs &a, const At &at, const float (&acc)[4][8], void *out, float *part,
                                         int64_t ld) {
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int i = ty + 16 * r, d = tx + 16 * c;
            if (i >= at.len || d >= a.Dk) continue;
            if (part) part[((at.seq + i) * a.H + at.h) * a.Dk + d] = acc[r][c];
            else static_cast<float *>(out)[(at.seq + i) * ld + at.hk * a.Dk + d] = acc[r][c];
        }
}

// Pass 3 of the backward pass.
__global__ __launch_bounds__(256) void k_lin_grad(const LinArgs a) {
    extern __shared__ float sm[];
    float *Q = sm, *K = Q + LC * LP, *V = K + LC * LP, *W = V + LC * LP, *S = W + LC * LP, *P = S + 128 * LP;
    __shared__ LinDecay<LC> D;
    __shared__ float fs[LC], cs[LC], rs[LC], zs[8];
    const At at(a);
    load_tile(Q, LP, row<float>(a.q, at.seq, a.ldq, at.hk, a.Dk), a.ldq, a.Dk, at.len);
    load_tile(K, LP, row<float>(a.k, at.seq, a.ldk, at.hk, a.Dk), a.ldk, a.Dk, at.len);
    load_tile(V, LP, row<float>(a.v, at.seq, a.ldv, at.h, a.Dv), a.ldv, a.Dv, at.len);
    load_tile(W, LP, row<float>(a.go, at.seq, a.ldo, at.h, a.Dv), a.ldo, a.Dv, at.len);
    load_state(S, LP, a.S + at.state(a), a.Dk, a.Dv);
    if (threadIdx.x < 32) D.fill(a.g + at.seq * a.H + at.h, a.H, at.len);
    loaded();
    scale_tile(W, LP, a.Dv, a.scale);
    __syncthreads();
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;

    // R_ij = D_ij (w_i . v_j), P_ij = D_ij (q_i . k_j); row and column sums of W = R (q . k)
    float p[4][4] = {}, x[4][4] = {};
    mm<4, 4, LP, 1, 1, LP>(p, Q, K, a.Dk, LC);
    mm<4, 4, LP, 1, 1, LP>(x, W, V, a.Dv, LC);
    float col[4] = {};
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int i = ty + 16 * r, j = tx + 16 * c;
            const float d = j <= i ? D.pair(i, j) : 0.f;
            x[r][c] = j <= i ? x[r][c] * d : 0.f;
            const float w = j < i ? x[r][c] * p[r][c] : 0.f;
            p[r][c] = j <= i ? p[r][c] * d : 0.f;
            sum += w;
            col[c] += w;
        }
        sum = row_sum(sum);
        if (tx == 0) rs[ty + 16 * r] = sum;
    }
    // column sums over the 16 thread rows, in a fixed order, through P
#pragma unroll
    for (int c = 0; c < 4; ++c) P[ty * PP + tx + 16 * c] = col[c];
    __syncthreads();
    if (threadIdx.x < LC) {
        float s = 0.f;
        for (int y = 0; y < 16; ++y) s += P[y * PP + threadIdx.x];
        rs[threadIdx.x] -= s;
    }
    __syncthreads();
    // dq
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) P[(ty + 16 * r) * PP + tx + 16 * c] = x[r][c];
    {
        float acc[4][8] = {};
        mm<4, 8, LP, 1, 1, LP>(acc, W, S, a.Dv, a.Dk);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = ty + 16 * r;
            const float f = D.first(i);
            float dot = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                acc[r][c] *= f;
                if (tx + 16 * c < a.Dk) dot = fmaf(acc[r][c], Q[i * LP + tx + 16 * c], dot);
            }
            dot = row_sum(dot);
            if (tx == 0) fs[i] = dot;
        }
        __syncthreads();        // P holds R
        mm<4, 8, PP, 1, LP, 1>(acc, P, K, LC, a.Dk);
        put_grad(a, at, acc, a.dq, a.pq, a.ldq);
    }
    // <Z, S>, then Z in S's place
    {
        const float *Z = a.dS + at.state(a);
        const int n4 = a.Dv >> 2;
        float dot = 0.f;
        for (int i = threadIdx.x; i < a.Dk * n4; i += 256) {
            const int d = i / n4, e = (i - d * n4) << 2;
            float4 *s = reinterpret_cast<float4 *>(S + d * LP + e);
            const float4 z = *reinterpret_cast<const float4 *>(Z + int64_t(d) * a.Dv + e), y = *s;
            dot += z.x * y.x + z.y * y.y + z.z * y.z + z.w * y.w;
            *s = z;             // every thread of the block is past its reads of S (the barrier above)
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(~0u, dot, d);
        if ((threadIdx.x & 31) == 0) zs[threadIdx.x >> 5] = dot;
        __syncthreads();
    }
    // dk
    {
        float acc[4][8] = {};
        mm<4, 8, LP, 1, 1, LP>(acc, V, S, a.Dv, a.Dk);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int j = ty + 16 * r;
            const float l = D.last(j);
            float dot = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                acc[r][c] *= l;
                if (tx + 16 * c < a.Dk) dot = fmaf(acc[r][c], K[j * LP + tx + 16 * c], dot);
            }
            dot = row_sum(dot);
            if (tx == 0) cs[j] = dot;
        }
        mm<4, 8, 1, PP, LP, 1>(acc, P, Q, LC, a.Dk);
        put_grad(a, at, acc, a.dk, a.pk, a.ldk);
    }
    __syncthreads();            // P is free, cs is written
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) P[(ty + 16 * r) * PP + tx + 16 * c] = p[r][c];
    // dv
    {
        float acc[4][8] = {};
        mm<4, 8, LP, 1, LP, 1>(acc, K, S, a.Dk, a.Dv);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float l = D.last(ty + 16 * r);
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[r][c] *= l;
        }
        __syncthreads();
        mm<4, 8, 1, PP, LP, 1>(acc, P, W, LC, a.Dv);
        float *dv = static_cast<float *>(a.dv) + at.seq * a.ldv + at.h * a.Dv;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int j = ty + 16 * r, e = tx + 16 * c;
                if (j < at.len && e < a.Dv) dv[j * a.ldv + e] = acc[r][c];
            }
    }
    // dg
    if (threadIdx.x < LC) {
        const int t = threadIdx.x;
        float across = 0.f, reads = 0.f, inside = 0.f;
        for (int w = 0; w < 8; ++w) across += zs[w];
        across *= D.total();
        for (int j = 0; j < t; ++j) across += cs[j];
        for (int i = LC - 1; i >= t; --i) {
            reads += fs[i];
            inside += rs[i];
        }
        const int64_t n = (at.seq + t) * a.H + at.h;
        if (t < at.len) {
            const bool cut = t ? D.r[t] != D.r[t - 1] : D.r[0] != 0;
            // no pair of the chunk crosses its first token
            a.dg[n] = cut ? 0.f : across + reads + (t ? inside : 0.f);
        }
    }
}

// Shared heads: out[token][hk][d] = sum over the group's heads of part[token][h][d].
template <class T>
__global__ __launch_bounds__(256) void k_lin_share(const LinArgs a) {
    const int n4 = a.Dk >> 2, rep = a.H / a.Hk;
    const int64_t n = a.B * a.T * a.Hk * n4;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
        const int d = int(i % n4) << 2;
        const int64_t r = i / n4, hk = r % a.Hk, tok = r / a.Hk;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const float *p = (w ? a.pk : a.pq) + (tok * a.H + hk * rep) * a.Dk + d;
            float4 s = f4(0.f);
            for (int h = 0; h < rep; ++h) s = s + ld_stream4(p + int64_t(h) * a.Dk);
            st4(static_cast<T *>(w ? a.dk : a.dq) + tok * (w ? a.ldk : a.ldq) + hk * a.Dk + d, s);
        }
    }
}

// The step.  A block owns `cols` state columns (a multiple of 4) of one sequence's head;
// thread (rg, cg) carries four columns of the rows rg, rg + RG, ...: S <- a S + k v^T and its
// part of q S, whose sum over rg is taken through shared memory.  Bound by the state's 8 Dk Dv
// bytes: 256 sequences x 16 heads of 128 take 80.5 us, 0.98 of the copy bandwidth.  Columns are
// split further when there are few heads, to use more SMs (one sequence: 2.9 us).
template <class T>
__global__ __launch_bounds__(256) void k_lin_step(const LinArgs a, float *__restrict__ state, int64_t n_slots,
                                                  const int32_t *__restrict__ slots, int cols) {
    __shared__ float q[128], k[128];
    __shared__ float4 part[256];
    const int64_t bh = blockIdx.x, b = bh / a.H, h = bh - b * a.H, hk = h / (a.H / a.Hk);
    const int e0 = blockIdx.y * cols, w4 = min(cols, a.Dv - e0) >> 2, RG = 256 / w4;
    const int cg = threadIdx.x % w4, rg = threadIdx.x / w4;
    const int64_t slot = slots ? slots[b] : b;
    T *o = static_cast<T *>(a.o) + b * a.ldo + h * a.Dv + e0 + 4 * cg;
    if (slot < 0 || slot >= n_slots) {
        if (rg == 0) st4(o, f4(0.f));
        return;
    }
    float *S = state + ((slot * a.H + h) * a.Dk) * a.Dv + e0 + 4 * cg;
    constexpr int U = 8;
    float4 s[U];
    if (rg < RG)
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (rg + u * RG < a.Dk) s[u] = *reinterpret_cast<const float4 *>(S + int64_t(rg + u * RG) * a.Dv);
    const float decay = expf(a.g[b * a.H + h]);
    if (threadIdx.x < a.Dk) {
        q[threadIdx.x] = float(row<T>(a.q, b, a.ldq, hk, a.Dk)[threadIdx.x]) * a.scale;
        k[threadIdx.x] = float(row<T>(a.k, b, a.ldk, hk, a.Dk)[threadIdx.x]);
    }
    float v[4];
    ld4(row<T>(a.v, b, a.ldv, h, a.Dv) + e0 + 4 * cg, v);
    __syncthreads();
    float4 acc = f4(0.f);
    if (rg < RG) {
        const float4 vv = make_float4(v[0], v[1], v[2], v[3]);
        for (int d0 = rg; d0 < a.Dk; d0 += U * RG) {
            if (d0 != rg)
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (d0 + u * RG < a.Dk) s[u] = *reinterpret_cast<const float4 *>(S + int64_t(d0 + u * RG) * a.Dv);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int d = d0 + u * RG;
                if (d >= a.Dk) break;
                // a decay of zero drops the old state whatever it holds
                s[u] = decay == 0.f ? f4(k[d]) * vv : fma4(f4(decay), s[u], f4(k[d]) * vv);
                *reinterpret_cast<float4 *>(S + int64_t(d) * a.Dv) = s[u];
                acc = fma4(f4(q[d]), s[u], acc);
            }
        }
    }
    part[threadIdx.x] = acc;
    __syncthreads();
    if (rg == 0) {
        for (int r = 1; r < RG; ++r) acc = acc + part[r * w4 + cg];
        st4(o, acc);
    }
}

constexpr size_t SM_GRAD = size_t(4 * LC * LP + 128 * LP + LC * PP) * 4;

template <bool REV>
cudaError_t states(const LinArgs &a, cudaStream_t st) {
    {
        ProfScope ps(K_LIN_STATE, st);
        const size_t smem = size_t(LC) * (pitch_of(a.Dk) + pitch_of(a.Dv)) * 4 + 256;
        LIN_CUDA(allow_smem<k_lin_chunk_state<REV>>());
        k_lin_chunk_state<REV><<<dim3(unsigned(a.NC), a.H, unsigned(a.B)), 256, smem, st>>>(a);
        LIN_CUDA(cudaGetLastError());
    }
    return launch_lin_scan(a, a.NC, REV ? 2 : 1, st);
}

cudaError_t fwd_f32(const LinArgs &a, cudaStream_t st) {
    LIN_CUDA(states<false>(a, st));
    ProfScope ps(K_LIN_OUT, st);
    const size_t smem = (size_t(LC + a.Dk) * pitch_of(a.Dv) + LC * (pitch_of(a.Dk) + std::max(pitch_of(a.Dk), PP))) * 4;
    LIN_CUDA(allow_smem<k_lin_out>());
    k_lin_out<<<dim3(unsigned(a.NC), a.H, unsigned(a.B)), 256, smem, st>>>(a);
    return cudaGetLastError();
}

cudaError_t bwd_f32(const LinArgs &a, cudaStream_t st) {
    LIN_CUDA(states<false>(a, st));
    LIN_CUDA(states<true>(a, st));
    ProfScope ps(K_LIN_GRAD, st);
    LIN_CUDA(allow_smem<k_lin_grad>());
    k_lin_grad<<<dim3(unsigned(a.NC), a.H, unsigned(a.B)), 256, SM_GRAD, st>>>(a);
    return cudaGetLastError();
}

template <class T>
cudaError_t share(const LinArgs &a, cudaStream_t st) {
    ProfScope ps(K_LIN_SHARE, st);
    const int64_t n = lin_div(a.B * a.T * a.Hk * (a.Dk / 4), 256);
    k_lin_share<T><<<unsigned(std::min<int64_t>(n, 152 * 16)), 256, 0, st>>>(a);
    return cudaGetLastError();
}

inline size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

cudaError_t launch_lin_scan(const LinArgs &a, int64_t n, int dirs, cudaStream_t st) {
    ProfScope ps(K_LIN_SCAN, st);
    const int64_t half = lin_div(int64_t(a.Dk) * a.Dv, 512) * a.B * a.H;
    k_lin_scan<<<unsigned(half * (dirs == 3 ? 2 : 1)), 128, 0, st>>>(a, n, half, dirs == 2);
    return cudaGetLastError();
}

static size_t carve(LinArgs &a, bool bwd, bool bf16, char *base) {
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char *p = base ? base + off : nullptr;
        off += al256(bytes);
        return p;
    };
    auto floats = [&](size_t n) { return reinterpret_cast<float *>(take(n * 4)); };
    auto halves = [&](size_t n) { return reinterpret_cast<__nv_bfloat16 *>(take(n * 2)); };
    const int64_t heads = a.B * a.H, n = heads * (bf16 ? lin_split(a, bwd).nseg : a.NC);
    const size_t dd = size_t(a.Dk) * a.Dv;
    a.S = floats(n * dd);
    a.tot = floats(n);
    a.dS = a.dtot = a.pq = a.pk = nullptr;
    a.shi = a.slo = a.s3 = a.zhi = a.zlo = a.z3 = nullptr;
    if (bwd) {
        a.dS = floats(n * dd);
        a.dtot = floats(n);
        if (bf16) {
            const size_t chunks = size_t(heads) * a.NC, all = chunks * dd;
            const size_t third = chunks * lin_pieces(a.Dv) * 32 * a.Dk;
            a.shi = halves(all);
            a.slo = halves(all);
            a.s3 = halves(third);
            a.zhi = halves(all);
            a.zlo = halves(all);
            a.z3 = halves(third);
        }
        if (a.Hk < a.H) {
            a.pq = floats(size_t(a.B * a.T) * a.H * a.Dk);
            a.pk = floats(size_t(a.B * a.T) * a.H * a.Dk);
        }
    }
    return off;
}

size_t lin_ws_bytes(const LinArgs &a, bool bwd, bool bf16) {
    LinArgs t = a;
    return carve(t, bwd, bf16, nullptr);
}
void lin_ws_carve(LinArgs &a, bool bwd, bool bf16, void *base) { carve(a, bwd, bf16, static_cast<char *>(base)); }

cudaError_t launch_lin_fwd(const LinArgs &a, bool bf16, unsigned *status, cudaStream_t st) {
    if (a.NC == 0) return launch_lin_scan(a, 0, 1, st);      // s1 = s0
    return bf16 ? launch_lin_tc_fwd(a, status, st) : fwd_f32(a, st);
}
cudaError_t launch_lin_bwd(const LinArgs &a, bool bf16, unsigned *status, cudaStream_t st) {
    if (a.NC == 0) return launch_lin_scan(a, 0, 2, st);       // ds0 = ds1
    LIN_CUDA(bf16 ? launch_lin_tc_bwd(a, status, st) : bwd_f32(a, st));
    if (!a.pq) return cudaSuccess;
    return bf16 ? share<__nv_bfloat16>(a, st) : share<float>(a, st);
}
cudaError_t launch_lin_step(const LinArgs &a, bool bf16, float *state, int64_t n_slots, const int32_t *slots,
                            cudaStream_t st) {
    ProfScope ps(K_LIN_STEP, st);
    int cols = a.Dv;
    while (cols % 8 == 0 && cols > 32 && a.B * a.H * lin_div(a.Dv, cols) < 152) cols /= 2;
    const dim3 grid(unsigned(a.B * a.H), unsigned(lin_div(a.Dv, cols)));
    if (bf16) k_lin_step<__nv_bfloat16><<<grid, 256, 0, st>>>(a, state, n_slots, slots, cols);
    else k_lin_step<float><<<grid, 256, 0, st>>>(a, state, n_slots, slots, cols);
    return cudaGetLastError();
}

}  // namespace adj
