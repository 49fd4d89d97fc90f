// Tensor-core and copy helpers of the latent-attention kernels, on top of
// sm100_ptx.cuh: products whose first operand is in tensor memory, tensor
// maps over packed rows, and waits that end when any role of the CTA failed.
#pragma once

#include <cuda.h>

#include "kda_latent.cuh"
#include "sm100_ptx.cuh"

namespace kda {

// Shared-memory operand descriptor in two words (sm100_ptx.cuh: smem_desc).
// A later k-step or slab of the same tile only adds to the address field of
// `lo`: one addition a product.  With the descriptor built anew for each, the
// issuing warp's dependent integer instructions took longer than the products
// (forward, B=4 T=8192 H=16: 1087 us).
struct Desc {
    uint32_t lo, hi;
    __device__ __forceinline__ Desc operator+(uint32_t sixteenths) const { return {lo + sixteenths, hi}; }
};
// K-major operand of 128-byte swizzled slabs (64 columns each); the k-step
// (16 columns) ks of a slab is + 2 ks.
__device__ __forceinline__ Desc desc_k(uint32_t saddr) {
    return {((saddr & 0x3FFFFu) >> 4) | (1u << 16), (1024u >> 4) | (1u << 14) | ((uint32_t)SW_128B << 29)};
}
// The same slabs as an MN-major operand (their rows are the k axis), `rows`
// rows each; k-step ks, rows 16 ks .. 16 ks + 15, is + 128 ks.
__device__ __forceinline__ Desc desc_mn(uint32_t saddr, uint32_t rows) {
    return {((saddr & 0x3FFFFu) >> 4) | ((rows * 128u >> 4) << 16),
            (1024u >> 4) | (1u << 14) | ((uint32_t)SW_128B << 29)};
}

// D[tmem] (+)= A[smem] B[smem]; whole converged warp, one elected lane issues.
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, Desc a, Desc b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]: rows of A in the lanes, two 16-bit elements
// of a row in each 32-bit column, the even one in the low half.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, Desc b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\t.reg .b64 db;\n\t"
        "mov.b64 db, {%2, %3};\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two 32-bit operations in one instruction: (a, b) c + d, and (a, b) + (c, d).
__device__ __forceinline__ void fma2(float& a, float& b, float c, float d) {
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d));
}
__device__ __forceinline__ void add2(float& a, float& b, float c, float d) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d));
}
// Of three (NaN only from three NaN).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float m;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}
// The largest of 32 values, in four independent chains.
__device__ __forceinline__ float max32(const float (&x)[32]) {
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = fmaxf(x[i], x[i + 4]);
#pragma unroll
    for (int e = 8; e < 32; e += 8)
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = max3(m[i], x[e + i], x[e + i + 4]);
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
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

// 16 lanes x 64 columns: thread i < 16 gets columns 0-31 of lane i, thread
// 16 + i columns 32-63 of it (an M = 64 product fills 16 of a warp's 32 lanes).
__device__ __forceinline__ void tmem_ld_half32(uint32_t taddr, float (&r)[32]) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32], 32;"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
          "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
          "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]),
          "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]),
          "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr)
        : "memory");
}

// Result tiles go through shared memory (slabs of 64 16-bit columns x 128
// rows, 16-byte pieces swizzled by the row): a thread has a whole row, and
// rows written straight to global memory are 32 lines an instruction (a
// 128 x 192 tile 6000 cycles beside about 1500).
__device__ __forceinline__ uint8_t* staged(uint8_t* slabs, int row, int piece) {
    return slabs + (piece >> 3) * (LAT_TILE * 128) + row * 128 + (((piece & 7) ^ (row & 7)) * 16);
}
// Rows [0, rows) of PIECES 16-byte pieces to out, `stride` bytes apart.
template <int PIECES>
__device__ __forceinline__ void copy_rows(uint8_t* slabs, void* out, long long stride, int rows, int tid, int threads) {
    for (int i = tid; i < rows * PIECES; i += threads) {
        const int r = i / PIECES, c = i % PIECES;
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) + r * stride + c * 16) =
            *reinterpret_cast<const uint4*>(staged(slabs, r, c));
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

// The same for a converged warp, every lane polling, joined by a vote: the
// compiler knows a vote's result to be uniform and keeps the operands of the
// products behind it in uniform registers.  (One lane polling in a branch of
// its own loses that: forward at B=4 T=8192 H=16 5.3 ms instead of 1.02; one
// elected lane polling, 1.06.)
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, uint32_t limit, volatile uint32_t* failed) {
    return __all_sync(0xffffffffu, wait_phase(bar, parity, limit, failed));
}

// ---- clusters: the CTA's place, a barrier of all threads, another CTA's shared memory ----
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(uint32_t saddr, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    return a;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// Tensor map over packed rows: [tokens][heads][width] 16-bit elements, rows
// `row_stride` elements apart (and heads `head_stride`, width where it is 0),
// boxes of 64 columns of one head and `box_rows` rows, 128-byte swizzled; rows
// past the end read as zero.
bool latent_row_map(CUtensorMap* m, const void* base, int width, int heads, long long tokens, long long row_stride,
                    int box_rows, long long head_stride = 0);

}  // namespace kda
