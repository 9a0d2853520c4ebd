// adj_tc5.cuh -- tcgen05 building blocks of the linear-attention kernels: bf16 tiles in the
// 128-byte swizzle, both operand orders, operand A from shared or tensor memory, and
// tensor-memory loads and stores of one warp's 32 lanes.
//
// A tile of R rows by W columns (64 or 128) of bf16 is stored as W / 64 panels of R rows by
// 128 bytes; the 16-byte unit u of row r lies at r * 128 + ((u ^ (r & 7)) << 4) of its panel.
// Read along its rows (K-major) or across them (MN-major) by the choice of descriptor.
#pragma once
#include <cuda.h>

#include "adj_ptx.cuh"
#include "adj_tmap.cuh"

namespace adj {
namespace tc5 {

// byte offset of unit u (8 values) of row r; panel: bytes of one panel
__device__ __forceinline__ uint32_t unit_at(int r, int u, uint32_t panel) {
    return uint32_t(u >> 3) * panel + uint32_t(r) * 128u + (uint32_t((u ^ r) & 7) << 4);
}

// rows are M or N, K runs along a row
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {
    return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
           (uint64_t(2) << 61);
}
// rows are K, M or N runs along a row; panel: distance of the 64-column panels; rows8: of 8-row groups
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t panel, uint32_t rows8 = 1024) {
    return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t(panel >> 4) << 16) | (uint64_t(rows8 >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// rows of 32 values in the 64-byte swizzle, K along a row: unit u of row r lies at r * 64 + ((u ^ (r >> 1) & 3) << 4)
__device__ __forceinline__ uint64_t desc_k64(uint32_t saddr) {
    return uint64_t((saddr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) | (uint64_t(512 >> 4) << 32) | (uint64_t(1) << 46) |
           (uint64_t(4) << 61);
}
// bf16 x bf16 -> fp32, M = 128
__device__ __forceinline__ uint32_t idesc(int n, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) | (uint32_t(n >> 3) << 17) |
           (uint32_t(128 >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(uint32_t(acc))
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(uint32_t(acc))
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// One operand in shared memory: where it starts, the bytes of a panel, and whether K runs
// across the rows.  The descriptor of k-step ks (16 of K) is the first one's plus an offset.
struct Tile {
    uint32_t at, panel;
    bool mn;
    __device__ __forceinline__ uint64_t first() const { return mn ? desc_mn(at, panel) : desc_k(at); }
    __device__ __forceinline__ uint64_t step(int ks) const {
        return uint64_t((mn ? uint32_t(ks) * 2048u : uint32_t(ks >> 2) * panel + uint32_t(ks & 3) * 32u) >> 4);
    }
};
// D[128, N] (+)= A B over K16 steps of 16
template <int N, int K16, bool A_MN, bool B_MN>
__device__ __forceinline__ void product(uint32_t d, uint32_t a, uint32_t a_panel, uint32_t b, uint32_t b_panel, bool acc) {
    const Tile ta{a, a_panel, A_MN}, tb{b, b_panel, B_MN};
    const uint64_t da = ta.first(), db = tb.first();
#pragma unroll
    for (int k = 0; k < K16; ++k) mma_ss(d, da + ta.step(k), db + tb.step(k), idesc(N, A_MN, B_MN), acc || k);
}
// the same over 32 of K, with B [N][32] in the 64-byte swizzle
template <int N>
__device__ __forceinline__ void product32(uint32_t d, uint32_t a, uint32_t b, bool acc) {
    const uint64_t da = desc_k(a), db = desc_k64(b);
#pragma unroll
    for (int k = 0; k < 2; ++k) mma_ss(d, da + uint64_t(2 * k), db + uint64_t(2 * k), idesc(N, false, false), acc || k);
}
// A in tensor memory: bf16 pairs, 8 columns a step; B across its rows
template <int N, int K16>
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t b_panel, bool acc) {
    const Tile tb{b, b_panel, true};
    const uint64_t db = tb.first();
#pragma unroll
    for (int k = 0; k < K16; ++k) mma_ts(d, a + uint32_t(k) * 8u, db + tb.step(k), idesc(N, false, true), acc || k);
}

// A in tensor memory as sums of two bf16, in the columns of the fp32 values that they come from: of
// every 8 columns the first four hold the values rounded down to bf16, the others what that lost.  A
// step of 16 takes the same 8 rows of B twice: its 8-row groups lie a distance of zero apart.
template <int N, int K8>
__device__ __forceinline__ void product_ts2(uint32_t d, uint32_t a, uint32_t b, uint32_t b_panel) {
    const uint64_t db = desc_mn(b, b_panel, 0u);
#pragma unroll
    for (int k = 0; k < K8; ++k) mma_ts(d, a + uint32_t(k) * 8u, db + uint64_t(k * 64), idesc(N, false, true), k != 0);
}

// Columns of one warp's 32 lanes: thread t gets those of lane t.  The wait is part of the load,
// so that no use of a register can come before it.
__device__ __forceinline__ void ld8(uint32_t t, float (&v)[8]) {
    uint32_t r[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(t)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void ld16(uint32_t t, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// two loads in flight
__device__ __forceinline__ void ld16x2(uint32_t t, uint32_t u, float (&v)[16], float (&w)[16]) {
    uint32_t r[16], q[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]), "=r"(q[7]), "=r"(q[8]), "=r"(q[9]), "=r"(q[10]), "=r"(q[11]), "=r"(q[12]), "=r"(q[13]), "=r"(q[14]), "=r"(q[15])
        : "r"(t), "r"(u)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        v[i] = __uint_as_float(r[i]);
        w[i] = __uint_as_float(q[i]);
    }
}
__device__ __forceinline__ void st4(uint32_t t, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(t), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ void st8(uint32_t t, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void alloc512(uint32_t *slot) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void free512(uint32_t tmem) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// x is a multiple of 64 values: every box starts on a 16-byte boundary
__device__ __forceinline__ void load4(uint32_t dst, const CUtensorMap *m, int x, int head, int t, int b, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(head), "r"(t), "r"(b), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void store4(const CUtensorMap *m, int x, int head, int t, int b, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(x), "r"(head), "r"(t), "r"(b), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void store3(const CUtensorMap *m, int x, int y, int z, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void load3(uint32_t dst, const CUtensorMap *m, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}


__device__ __forceinline__ uint32_t pack(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&v);
}
// the upper 16 bits of two values: bf16 by truncation, in one instruction where the rounding
// conversion takes four issue slots.  For the parts of a sum, whose remainder the next part takes
// up, it serves as well.
__device__ __forceinline__ uint32_t pack_top(float a, float b) {
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float top(float a) { return __uint_as_float(__float_as_uint(a) & 0xFFFF0000u); }
// 8 values as sums of two bf16, for product_ts2
__device__ __forceinline__ void split8(const float (&p)[8], uint32_t (&r)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        r[e] = pack_top(p[2 * e], p[2 * e + 1]);
        r[4 + e] = pack_top(p[2 * e] - top(p[2 * e]), p[2 * e + 1] - top(p[2 * e + 1]));
    }
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint4 lds(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
// 32 bytes to global memory, on 32
__device__ __forceinline__ void stg32(void *p, uint4 a, uint4 b) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x),
                 "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}
__device__ __forceinline__ void sts(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// [B, T, heads, D] bf16 with token pitch ld: boxes of 64 values x 1 head x `rows` tokens
inline bool map_tokens(CUtensorMap *m, const void *p, int64_t D, int64_t heads, int64_t T, int64_t B, int64_t ld,
                       int rows = 128) {
    auto enc = tmap_encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {cuuint64_t(D), cuuint64_t(heads), cuuint64_t(T), cuuint64_t(B)};
    const cuuint64_t strides[3] = {cuuint64_t(D) * 2, cuuint64_t(ld) * 2, cuuint64_t(T * ld) * 2};
    const cuuint32_t box[4] = {64, 1, cuuint32_t(rows), 1}, one[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// [n, Dk, Dv] bf16, dense: boxes of 64 columns x `rows` rows of one matrix
inline bool map_states(CUtensorMap *m, const void *p, int64_t Dv, int64_t Dk, int64_t n, int rows) {
    auto enc = tmap_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {cuuint64_t(Dv), cuuint64_t(Dk), cuuint64_t(n)};
    const cuuint64_t strides[2] = {cuuint64_t(Dv) * 2, cuuint64_t(Dk * Dv) * 2};
    const cuuint32_t box[3] = {64, cuuint32_t(rows), 1}, one[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// [n, pieces, Dk, 32] bf16, dense: boxes of one piece, `rows` rows of it, in the 64-byte swizzle
inline bool map_pieces(CUtensorMap *m, const void *p, int64_t Dk, int64_t pieces, int64_t n, int rows) {
    auto enc = tmap_encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {32, cuuint64_t(Dk), cuuint64_t(pieces), cuuint64_t(n)};
    const cuuint64_t strides[3] = {64, cuuint64_t(Dk) * 64, cuuint64_t(Dk * pieces) * 64};
    const cuuint32_t box[4] = {32, cuuint32_t(rows), 1, 1}, one[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc5
}  // namespace adj
