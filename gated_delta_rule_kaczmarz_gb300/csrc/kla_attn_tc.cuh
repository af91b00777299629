// What the tensor-core attention kernels share: tiles of packed rows, tensor
// maps, descriptors and the packed fp32 instructions of the softmax.
#pragma once

#include "kla_attn.cuh"
#include "kla_tc.cuh"
#include "kla_tmap.h"

namespace kla {
namespace attn {

constexpr int kTile = 128;               // rows and keys of a tile
constexpr uint32_t kSlab = 128 * 128;    // bytes of 128 rows x 64 features, 128-byte swizzle

// Tokens of a tile whose rows are token x group head.
inline int tile_tokens(int G) { return kTile / G; }

// [rows][H][d] bf16 with row_stride elements between rows, as {feature, head,
// row}: box 64 features x `heads` heads x `rows_box` rows, so that box rows
// land in shared memory as (row, head) packed rows.
inline bool map_rows(CUtensorMap *m, const void *base, int d, int H, long rows,
                     long long row_stride, int heads, int rows_box) {
    if (tmap::encode_fn() == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)row_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)rows_box};
    const cuuint32_t es[3] = {1, 1, 1};
    return tmap::encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base),
                             dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

#ifdef __CUDACC__
// Operand of a product over features: K step ks of a tile's 64-feature slabs.
__device__ __forceinline__ uint64_t kdesc(uint32_t base, int ks) {
    return tc::sdesc_sw128(base + (uint32_t)(ks >> 2) * kSlab + (uint32_t)(ks & 3) * 32u, 16, 1024);
}
// Operand of a product over a tile's rows (its features are the N side): K
// step ks of 16 rows.
__device__ __forceinline__ uint64_t mdesc(uint32_t base, int ks) {
    return tc::sdesc_sw128(base + (uint32_t)ks * 2048u, kSlab, 1024);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
// A warpgroup's registers per thread (the kernel's launch has 168 each).
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// (x0, x1) * a + b, two at a time.
__device__ __forceinline__ void fma2(float &x0, float &x1, float a, float b) {
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "+f"(x0), "+f"(x1)
        : "f"(a), "f"(b));
}
// (s0, s1) += (x0, x1)
__device__ __forceinline__ void add2(float &s0, float &s1, float x0, float x1) {
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "add.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "+f"(s0), "+f"(s1)
        : "f"(x0), "f"(x1));
}
// Two bf16 values, the first in the low half.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
                 ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
                 : "memory");
}

// 16 bf16 values of a row: a thread stores a row of its own, so each store is a
// sector of its own, and half of one without the 32-byte form (forward, B 4, T
// 2048, 16 + 4 heads of 128: 67 us against 70; backward, B 16, T 512: 117 against
// 126).  It is not taken where the tensor is only 16-byte aligned.
__device__ __forceinline__ void store16(__nv_bfloat16 *p, const uint32_t (&u)[8]) {
    if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]),
                     "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(u[0], u[1], u[2], u[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(u[4], u[5], u[6], u[7]);
    }
}

// Asks for a block of this launch that has not started: the answer lands in
// *answer (16 bytes of shared memory, 16-byte aligned) and completes 16 bytes
// on *bar.  Not asked again once the answer was that there is none.
__device__ __forceinline__ void ask_block(uint4 *answer, uint64_t *bar) {
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128"
        " [%0], [%1];" ::"r"(tc::smem_u32(answer)), "r"(tc::smem_u32(bar))
        : "memory");
}
// The block of an answer, or -1.
__device__ __forceinline__ int answered_block(const uint4 *answer) {
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t"
        "ld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t"
        "mov.b32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
        : "=r"(got), "=r"(x)
        : "r"(tc::smem_u32(answer))
        : "memory");
    return got ? (int)x : -1;
}

// Zeroes rows from..127 of a tile's slabs (one warp) and makes the writes
// visible to the tensor cores: rows behind a sequence's last are a
// neighbour's, and 0 times what they hold need not be 0.
template <int SLABS>
__device__ __forceinline__ void zero_rows(unsigned char *tile, int from, int lane) {
    const int words = (kTile - from) * 8;          // 16-byte words of a slab
#pragma unroll
    for (int s = 0; s < SLABS; ++s) {
        uint4 *p = reinterpret_cast<uint4 *>(tile + s * kSlab + from * 128);
        for (int i = lane; i < words; i += 32) p[i] = make_uint4(0, 0, 0, 0);
    }
    tc::fence_async_smem();
    __syncwarp();
}
#endif

}  // namespace attn

bool attn_tc_ready();
cudaError_t launch_attn_tc_fwd(const attn::Args &a, int d, int total_k, cudaStream_t s);
cudaError_t launch_attn_tc_bwd(const attn::Args &keys, const attn::Args &rows, int d, int total_k,
                               cudaStream_t s);

}  // namespace kla
