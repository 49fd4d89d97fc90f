// Tensor-core and copy helpers of the latent-attention kernels, on top of
// sm100_ptx.cuh: products whose first operand is in tensor memory, tensor
// maps over packed rows, and waits that end when any role of the CTA failed.
#pragma once

#include <cuda.h>

#include "kda_latent.cuh"
#include "sm100_ptx.cuh"

namespace kda {

// D[tmem] (+)= A[tmem] B[smem]: rows of A in the lanes, two 16-bit elements
// of a row in each 32-bit column, the even one in the low half.  Whole
// converged warp, one elected lane issues.
__device__ __forceinline__ void mma_f16_ts_warp(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// K-major operand of 128-byte swizzled slabs (`rows` rows of 64 columns
// each): the descriptor of its k-step (16 columns) ks.
__device__ __forceinline__ uint64_t desc_k(uint32_t base, uint32_t rows, int ks) {
    return smem_desc(base + (uint32_t)(ks >> 2) * rows * 128u + (uint32_t)(ks & 3) * 32u, 16u, 1024u, SW_128B);
}
// The same tile as an MN-major operand (its rows are the k axis): k-step ks
// is rows 16 ks .. 16 ks + 15.
__device__ __forceinline__ uint64_t desc_mn(uint32_t base, uint32_t rows, int ks) {
    return smem_desc(base + (uint32_t)ks * 2048u, rows * 128u, 1024u, SW_128B);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a, b -> one 32-bit word of two rounded 16-bit floats, a in the low half.
template <bool FP16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    uint32_t r;
    if constexpr (FP16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
template <bool FP16>
__device__ __forceinline__ float2 unpack2(uint32_t x) {
    if constexpr (FP16) {
        const __half2 h = *reinterpret_cast<const __half2*>(&x);
        return __half22float2(h);
    } else {
        return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    }
}

// Bounded wait on a barrier phase.  Runs out after `limit` polls, or soon
// after another role of the CTA has set the failure flag; sets the flag.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, uint32_t limit, volatile uint32_t* failed) {
    for (uint32_t i = 0; i < limit; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63u) == 63u && *failed) return false;
    }
    *failed = 1u;
    return false;
}

// Tensor map over packed rows: [tokens][heads][width] 16-bit elements, rows
// `row_stride` elements apart, boxes of 64 columns of one head and `box_rows`
// rows, 128-byte swizzled; rows past the end read as zero.
bool latent_row_map(CUtensorMap* m, const void* base, int width, int heads, long long tokens, long long row_stride,
                    int box_rows);

}  // namespace kda
