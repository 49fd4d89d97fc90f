// Expanded latent attention, backward, in four launches:
//   aux   D_i = dout_i . o_i and log2(e) lse_i of every query and head, laid
//         out as the key kernel reads them; in fp16 the sizes of dout and v
//   dq    one CTA for 128 queries of a head, over the keys:
//           S = Q K^T, dP = dO V^T, dS = P (dP - D), dQ += dS K
//   dkv   one CTA for 128 keys of a head, over the queries:
//           S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q
//   dpe   the shared positional key's gradient: the heads' parts, in order
// with P = exp(scale S - lse), recomputed in both middle kernels: that is
// 1152 instead of 832 multiply-adds a pair, but no gradient is summed through
// memory by more than one CTA, so nothing is atomic and equal inputs give
// equal bits.  All products are tcgen05 with 32-bit accumulators in tensor
// memory.  S and dP are read to registers as soon as they are complete, so
// that the next tile's can be issued; P and dS go back to tensor memory in
// 16 bits as first operands.  dS is kept without the factor `scale`, which
// the final dq and dk get in 32 bits.
//
// Both roundings make operands of the tensor cores (32-bit ones run at half the
// rate and twice the columns): bf16 gradients are off by 0.0024 of their norm,
// 0.0018 of that their own rounding and o's; what is summed is in 32 bits.
//
// Packed T=9192 H=32 (six lengths, causal), alone: aux 29 us, dq 360, dkv 466, dpe 15
// (fp16 46, 366, 475, 15); in all 860 us in a graph, 832 TFLOP/s of the 832
// multiply-adds a pair, 1152 of those done.  B=4 T=8192 H=16 3.26 ms in a few
// calls after a pause, 1520 done, and 3.49, 1420, at the power limit.  What is left is the first loads
// and last stores of CTAs with some twelve steps each, and in dq the waits for
// K.  Not better: dq with its own dout . o beside aux (944 us).
#include "kda_latent_mma.cuh"

namespace kda {

namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr uint32_t SLAB = 64 * LAT_TILE * 2;            // 128 rows x 64 columns
// Warps 0-7 elementwise (with sixteen, no faster: B=4 T=8192 H=16 3.55 ms
// beside 3.48), 8 and 9 products, 10 loads.  Two warps issue so that
// one's waits (about 90 cycles each even when they succeed at once) pass while
// the other's products run: 8 the scores and dP, 9 the gradients.
constexpr int BWD_THREADS = 352;
constexpr int QT = 64;                                  // queries of a dkv step
constexpr uint32_t HSLAB = 64 * QT * 2;                 // 64 rows x 64 columns

struct BwdMaps {
    CUtensorMap q, dout, kv, pe;                        // boxes of 128 rows
    CUtensorMap q64, dout64;                            // of 64 rows
};

// fp16 P of the key kernel carries a factor 2^8: at long lengths the weights
// themselves would fall into fp16's subnormal range (below 6e-5).
template <bool FP16> constexpr float P_SHIFT = FP16 ? 8.f : 0.f;

// dS = P (dP - D) is as small as dout times the weights, which fp16 alone
// cannot hold: with unit keys and queries, 2048 keys and dout of 1e-4 most of
// it is below 6e-5 (dk off by 1.5e-2 of its norm), and large dout can put it
// past 65504.  So fp16 dS carries a factor 2^k until dq and dk are scaled in
// 32 bits, from 2 max |dout_i| max |v_j| >= |dP - D| of the sequence and head
// (o is a mean of values): 2^k times that bound is in [2^13, 2^14), four times
// below fp16's end, and the typical dS of L keys near 2^9 / L.  (bf16 has
// fp32's range and k = 0.)  The two maxima (of squared norms, as bits; rows
// that are not finite and queries without keys do not count) wait in the
// sequence's rows of dk_pe, which the last launch writes and none reads: 16 lk
// pairs, so heads share one only where they are more than 16 times the keys.
__device__ __forceinline__ uint32_t* grad_sizes(const LatentParams& p, const LatentSeq& s, int h) {
    return static_cast<uint32_t*>(p.dk_pe) + s.k0 * (LAT_P / 2) + 2 * (h % min((long long)p.H, s.lk * (LAT_P / 4ll)));
}
template <bool FP16>
__device__ __forceinline__ int grad_shift(const LatentParams& p, const LatentSeq& s, int h) {
    if (!FP16 || s.lq == 0 || s.lk == 0) return 0;
    const uint2 w = __ldcg(reinterpret_cast<const uint2*>(grad_sizes(p, s, h)));
    const float bound = 2.f * sqrtf(__uint_as_float(w.x)) * sqrtf(__uint_as_float(w.y));   // 0, or 2^-47 to 2^41
    return bound > 0.f ? 13 - ((int)(__float_as_uint(bound) >> 23) - 127) : 0;
}
__device__ __forceinline__ float pow2(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

// The largest of the block's non-negative values into *to.
__device__ __forceinline__ void block_max(float x, float (&part)[8], uint32_t* to) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, m));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 8; ++w) x = fmaxf(x, part[w]);
        atomicMax(to, __float_as_uint(x));   // (its operands' order does not change a maximum)
    }
}

// Per 64-query tile slot and head: 64 of log2(e) lse - P_SHIFT (+infinity for
// rows past the end and rows without keys: their weights become 0), 64 of D.
// In fp16 the blocks from `slots` on take the norms of a 64-key tile's values.
template <bool FP16>
__global__ void __launch_bounds__(256) latent_aux_kernel(const __grid_constant__ LatentParams p, int slots) {
    __shared__ float part[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.y;
    if (blockIdx.x == 0 && h == 0) check_offsets(p, threadIdx.x, 256);
    int n, j;
    LatentSeq s;
    if (FP16 && (int)blockIdx.x >= slots) {
        if (!latent_find(p, p.cu_k, p.Tk, (int)blockIdx.x - slots, QT, n, j, s) || j * QT >= s.lk) return;
        float most = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = j * QT + 2 * (8 * k + warp) + (lane >> 4);
            float sq = 0.f;
            if (i < s.lk) {
                const uint4 a = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.kv) +
                                                               ((s.k0 + i) * p.H + h) * LAT_KV + LAT_N)[lane & 15];
                const uint32_t* x = &a.x;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 u = unpack2<FP16>(x[e]);
                    sq += u.x * u.x + u.y * u.y;
                }
            }
#pragma unroll
            for (int m = 8; m > 0; m >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, m);
            if (sq < INFINITY) most = fmaxf(most, sq);
        }
        block_max(most, part, grad_sizes(p, s, h) + 1);
        return;
    }
    if (!latent_find(p, p.cu_q, p.Tq, blockIdx.x, QT, n, j, s) || j * QT >= s.lq) return;
    float* aux = p.aux + ((long long)blockIdx.x * p.H + h) * 2 * QT;
    float most = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {                       // two rows a warp at a time, 16 bytes a lane
        const int r = 2 * (8 * k + warp) + (lane >> 4);
        const int i = j * QT + r;
        const long long row = (s.q0 + i) * p.H + h;
        float d = 0.f, sq = 0.f;
        if (i < s.lq) {
            const uint4 a = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.dout) + row * LAT_V)[lane & 15];
            const uint4 b = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.o) + row * LAT_V)[lane & 15];
            const uint32_t *x = &a.x, *y = &b.x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 u = unpack2<FP16>(x[e]), v = unpack2<FP16>(y[e]);
                d += u.x * v.x + u.y * v.y;
                if constexpr (FP16) sq += u.x * u.x + u.y * u.y;
            }
        }
#pragma unroll
        for (int m = 8; m > 0; m >>= 1) {
            d += __shfl_xor_sync(0xffffffffu, d, m);
            if constexpr (FP16) sq += __shfl_xor_sync(0xffffffffu, sq, m);
        }
        if ((lane & 15) == 0) {
            const float lse = i < s.lq ? p.lse[row] : -INFINITY;
            aux[r] = lse == -INFINITY ? INFINITY : lse * LOG2E - P_SHIFT<FP16>;
            aux[QT + r] = d;
            if (FP16 && lse != -INFINITY && sq < INFINITY) most = fmaxf(most, sq);
        }
    }
    if (FP16 && s.lk > 0) block_max(most, part, grad_sizes(p, s, h));
}

// Sixteen registers -> columns col .. col + 15 of this thread's lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) tmem_st4(taddr + i, r[i], r[i + 1], r[i + 2], r[i + 3]);
}

// ---------------------------------------------------------------------------
// dq.  Shared memory: Q and dO (five slabs), K through a ring of seven slabs,
// V through one of two.  K of step j is needed by S (j) and, most of a step
// later, by dQ (j), which frees it slab by slab: the first slab of K (j + 2)
// has a place of its own, the other two load behind the slabs of dQ (j).
// Tensor memory: S 128 columns, dP 128, dS 64 (16-bit), dQ 192: all 512.
// A step is 2050 cycles of products and takes about 2600 with its waits; a CTA
// (packed T=9192 H=32: 12 steps, 382 us in all) begins with 6000 cycles of
// setup and first loads.  Not better: three K stages by tiles of 96 keys (products of
// 96 columns run little faster than of 128: packed T=9192 H=32 449 us beside
// 390), or by dO in tensor memory with dS over dP (S (j + 1), dQ and dP then
// run one after another and nothing is left beside the elementwise part: 414
// us, with sixteen elementwise warps 432).
// ---------------------------------------------------------------------------
constexpr uint32_t KRING = 7;
constexpr uint32_t D_Q = 0, D_DO = 3 * SLAB, D_K = 5 * SLAB, D_V = D_K + KRING * SLAB, D_BAR = D_V + 2 * SLAB;
constexpr uint32_t D_QFULL = D_BAR, D_DOFULL = D_QFULL + 8, D_KFULL = D_DOFULL + 8 /* [2]: first slab */,
                   D_KREST = D_KFULL + 16 /* [second, third slab][2] */, D_VFULL = D_KREST + 32, D_SFULL = D_VFULL + 8,
                   D_PFULL = D_SFULL + 8, D_SREAD = D_PFULL + 8, D_PREAD = D_SREAD + 8, D_DSFULL = D_PREAD + 8,
                   D_DONE = D_DSFULL + 8 /* [3]: by step % 3 */, D_KFREE = D_DONE + 24 /* [slab 0, 1][3] */,
                   D_DRAIN = D_KFREE + 48, D_TMEM = D_DRAIN + 16, D_FAILED = D_TMEM + 4;
constexpr uint32_t D_SMEM = D_FAILED + 4 + 1024;
static_assert(D_SMEM <= 232448, "shared memory of one CTA");

template <bool FP16>
__global__ void __launch_bounds__(BWD_THREADS, 1)
    latent_dq_kernel(const __grid_constant__ LatentParams p, const __grid_constant__ BwdMaps maps, int slots) {
    // the tables are there; the key kernel, which needs nothing else of this launch, may start beside its end
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
    volatile uint32_t* failed = reinterpret_cast<volatile uint32_t*>(smem + D_FAILED);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t limit = p.wait_limit != 0u ? p.wait_limit : WAIT_LIMIT;

    int n, j0;
    LatentSeq s;
    int slot, h;
    latent_order(p, (int)blockIdx.x, slots, true, slot, h);
    const bool found = latent_find(p, p.cu_q, p.Tq, slot, LAT_TILE, n, j0, s);
    const int row0 = found ? j0 * LAT_TILE : 0;
    if (!found || row0 >= s.lq) {
        return;
    }
    const int shift = s.lk - s.lq;
    const int most = p.causal ? min(s.lk, min(row0 + LAT_TILE, s.lq) + shift) : s.lk;
    const int steps = most > 0 ? (most + LAT_TILE - 1) / LAT_TILE : 0;

    if (tid == 32) {
        prefetch_map(&maps.q);
        prefetch_map(&maps.kv);
        prefetch_map(&maps.pe);
        prefetch_map(&maps.dout);
    }
    if (tid == 0) {
        for (uint32_t i = 0; i < 6; ++i) mbar_init(base + D_KFULL + 8 * i, 1);
        mbar_init(base + D_VFULL, 1);
        mbar_init(base + D_QFULL, 1);
        mbar_init(base + D_DOFULL, 1);
        mbar_init(base + D_SFULL, 1);
        mbar_init(base + D_PFULL, 1);
        mbar_init(base + D_SREAD, 8);
        mbar_init(base + D_PREAD, 8);
        mbar_init(base + D_DSFULL, 8);
        for (uint32_t i = 0; i < 9; ++i) mbar_init(base + D_DONE + 8 * i, 1);
        mbar_init(base + D_DRAIN, 1);
        mbar_init(base + D_DRAIN + 8, 1);
        *failed = 0u;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(base + D_TMEM, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + D_TMEM);
    const uint32_t t_s = tmem, t_p = tmem + 128, t_ds = tmem + 256, t_dq = tmem + 320;

    if (warp == 10) {
        if (lane == 0 && steps > 0) {
            const int tq = (int)s.q0 + row0;
            mbar_arrive_expect_tx(base + D_QFULL, 3 * SLAB);
            for (uint32_t c = 0; c < 3; ++c) tma_load_3d(base + D_Q + c * SLAB, &maps.q, 64 * c, h, tq, base + D_QFULL);
            mbar_arrive_expect_tx(base + D_DOFULL, 2 * SLAB);
            // K slab i takes the place of slab i - 7: the first of step j that of K (j - 3)'s last, the others those of
            // K (j - 2)'s first two; dP (j - 1) frees V.  (A barrier waited for late must not get a phase ahead: what
            // dQ frees has three barriers in turn, the next use of one needs the K that is asked for here.)
            int a[3] = {0, 0, 0}, v = 0;   // K slabs and V tiles asked for
            bool ok = true;
            for (int j = 0; j < steps && ok; ++j) {
                const int tok = (int)s.k0 + j * LAT_TILE, st = j & 1;
                for (int c = 0; c < 3 && ok; ++c) {
                    const int of = c == 0 ? j - 3 : j - 2;   // the step whose slab goes
                    if (of >= 0)
                        ok = wait_phase(base + (c == 0 ? D_DONE : D_KFREE + 24 * (c - 1)) + 8 * (of % 3), (of / 3) & 1, limit,
                                        failed);
                    if (!ok) break;
                    const uint32_t bar = base + (c == 0 ? D_KFULL : D_KREST + 16 * (c - 1)) + 8 * st;
                    const uint32_t dst = base + D_K + (uint32_t)((3 * j + c) % KRING) * SLAB;
                    mbar_arrive_expect_tx(bar, SLAB);
                    if (c < 2) tma_load_3d(dst, &maps.kv, 64 * c, h, tok, bar);
                    else tma_load_3d(dst, &maps.pe, 0, 0, tok, bar);
                    ++a[c];
                }
                if (j == 0)
                    for (uint32_t c = 0; c < 2; ++c)
                        tma_load_3d(base + D_DO + c * SLAB, &maps.dout, 64 * c, h, tq, base + D_DOFULL);
                if (ok && j >= 1) ok = wait_phase(base + D_PFULL, (j - 1) & 1, limit, failed);
                if (!ok) break;
                mbar_arrive_expect_tx(base + D_VFULL, 2 * SLAB);
                for (uint32_t c = 0; c < 2; ++c)
                    tma_load_3d(base + D_V + c * SLAB, &maps.kv, LAT_N + 64 * c, h, tok, base + D_VFULL);
                ++v;
            }
            // every copy issued here has landed before the CTA ends
            mbar_wait(base + D_QFULL, 0, DRAIN_LIMIT);
            mbar_wait(base + D_DOFULL, 0, DRAIN_LIMIT);
            for (int c = 0; c < 3; ++c)
                for (int k = max(0, a[c] - 2); k < a[c]; ++k)
                    mbar_wait(base + (c == 0 ? D_KFULL : D_KREST + 16 * (c - 1)) + 8 * (k & 1), (k / 2) & 1, DRAIN_LIMIT);
            if (v > 0) mbar_wait(base + D_VFULL, (v - 1) & 1, DRAIN_LIMIT);
        }
    } else if (warp >= 8) {
        const MmaType ty = FP16 ? T_F16 : T_BF16;
        const uint32_t id = idesc_f16(ty, 128, 128, false, false), id64 = idesc_f16(ty, 128, 64, false, true);
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = ok && wait_warp(base + bar, parity, limit, failed);
            return ok;
        };
        auto score = [&](int j) {
#pragma unroll
            for (int c = 0; c < 3; ++c) {
                const uint32_t b = base + D_K + (uint32_t)((3 * j + c) % KRING) * SLAB;
                if (!wait((c == 0 ? D_KFULL : D_KREST + 16 * (c - 1)) + 8 * (j & 1), (j >> 1) & 1)) return;
                if ((j + 1) * LAT_TILE > s.lk) {
                    // rows past the sequence's end hold whatever follows: dS is 0 there and has to meet zeros
                    for (int r = s.lk - j * LAT_TILE + (lane >> 3); r < LAT_TILE; r += 4)
                        *reinterpret_cast<uint4*>(smem + (b - base) + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                    fence_async_smem();
                    __syncwarp();
                }
                const Desc da = desc_k(base + D_Q + c * SLAB), db = desc_k(b);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_ss(t_s, da + 2 * ks, db + 2 * ks, id, c + ks > 0);
            }
            mma_commit_warp(base + D_SFULL);
        };
        auto grad_p = [&](int j) {
            if (!wait(D_VFULL, j & 1)) return;
            const Desc da = desc_k(base + D_DO), db = desc_k(base + D_V);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                const uint32_t at = (ks >> 2) * (SLAB / 16) + (ks & 3) * 2;
                mma_ss(t_p, da + at, db + at, id, ks > 0);
            }
            mma_commit_warp(base + D_PFULL);
        };
        if (warp == 8) {
            if (steps > 0) {
                if (wait(D_QFULL, 0)) score(0);
                if (ok && wait(D_DOFULL, 0)) grad_p(0);
            }
            for (int j = 0; j + 1 < steps && ok; ++j) {
                if (!wait(D_SREAD, j & 1)) break;
                tc_fence_after();
                score(j + 1);
                if (!ok || !wait(D_PREAD, j & 1)) break;
                tc_fence_after();
                grad_p(j + 1);
            }
        } else {
            for (int j = 0; j < steps && wait(D_DSFULL, j & 1); ++j) {
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 3; ++c) {          // dQ += dS K, 64 of its columns a K slab
                    const Desc db = desc_mn(base + D_K + (uint32_t)((3 * j + c) % KRING) * SLAB, LAT_TILE);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) mma_ts(t_dq + 64 * c, t_ds + 8 * ks, db + 128 * ks, id64, j + ks > 0);
                    mma_commit_warp(base + (c < 2 ? D_KFREE + 24 * c : D_DONE) + 8 * (j % 3));
                }
            }
        }
        // every product issued here is done before the tensor memory is freed
        mma_commit_warp(base + D_DRAIN + 8 * (warp & 1));
        mbar_wait(base + D_DRAIN + 8 * (warp & 1), 0, DRAIN_LIMIT);
    } else {
        const int g = warp >> 2, row = row0 + (warp & 3) * 32 + lane;   // columns 64 g .. of S and dP
        const uint32_t quad = (uint32_t)(warp & 3) << 21;
        const float c = p.scale * LOG2E;
        const int kmax = p.causal ? min(s.lk, row + shift + 1) : s.lk;
        const bool there = row < s.lq;
        float lse2 = INFINITY, delta = 0.f;
        const int gs = grad_shift<FP16>(p, s, h);       // P here only makes dS: its factor is in lse2
        if (there) {   // the key kernel's tables: tile slot of 64 queries
            const int slot = p.cu_q == nullptr ? n * ((p.Tq + QT - 1) / QT) + row / QT : (int)(s.q0 / QT) + n + row / QT;
            const float* aux = p.aux + ((long long)slot * p.H + h) * 2 * QT + row % QT;
            lse2 = aux[0] + (P_SHIFT<FP16> - (float)gs);
            delta = aux[QT];
        }
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = ok && wait_warp(base + bar, parity, limit, failed);
            return ok;
        };
        for (int j = 0; j < steps; ++j) {
            if (!wait(D_SFULL, j & 1)) break;
            tc_fence_after();
            float x[2][32];
            tmem_ld32(t_s + 64 * g + quad, x[0]);
            tmem_ld32(t_s + 64 * g + 32 + quad, x[1]);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(base + D_SREAD);
            const int lim = kmax - j * LAT_TILE - 64 * g;
            const bool cut = __any_sync(0xffffffffu, lim < 64);
#pragma unroll
            for (int e = 0; e < 64; ++e) x[e >> 5][e & 31] = ex2(fmaf(x[e >> 5][e & 31], c, -lse2));
            if (!wait(D_PFULL, j & 1)) break;
            tc_fence_after();
            float w[32];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float d[32];
                tmem_ld32(t_p + 64 * g + 32 * b + quad, d);
                tmem_ld_wait();
                if (b == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(base + D_PREAD);
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) d[e] = x[b][e] * (d[e] - delta);
                if (cut) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) d[e] = 32 * b + e < lim ? d[e] : 0.f;
                }
#pragma unroll
                for (int e = 0; e < 32; e += 2) w[16 * b + (e >> 1)] = __uint_as_float(pack2<FP16>(d[e], d[e + 1]));
            }
            if (j > 0 && !wait(D_DONE + 8 * ((j - 1) % 3), ((j - 1) / 3) & 1)) break;   // dS is free
            tc_fence_after();
            tmem_st32(t_ds + 32 * g + quad, w);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(base + D_DSFULL);
        }
        if (steps > 0 && ok) wait(D_DONE + 8 * ((steps - 1) % 3), ((steps - 1) / 3) & 1);
        if (bar_and_named(1, 256, ok)) {
            // every product is done: Q's slabs take the result
            tc_fence_after();
            const int r = row - row0;
            const float undo = pow2(-gs);
#pragma unroll
            for (int b = 0; b < 3; ++b) {
                float d[32];
                if (steps > 0) {
                    tmem_ld32(t_dq + 96 * g + 32 * b + quad, d);
                    tmem_ld_wait();
                    if constexpr (FP16) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) d[e] *= undo;
                    }
                }
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = steps > 0 ? pack2<FP16>(d[e + 2 * k] * p.scale, d[e + 2 * k + 1] * p.scale) : 0u;
                    *reinterpret_cast<uint4*>(staged(smem + D_Q, r, 12 * g + 4 * b + (e >> 3))) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            bar_and_named(1, 256, true);
            copy_rows<LAT_QK / 8>(smem + D_Q, static_cast<uint16_t*>(p.dq) + ((s.q0 + row0) * p.H + h) * LAT_QK,
                                  (long long)p.H * LAT_QK * 2, min(LAT_TILE, s.lq - row0), tid, 256);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tmem, 512);
    if (tid == 0 && *failed) set_status(p.status, STATUS_TIMEOUT);
}

// ---------------------------------------------------------------------------
// dk, dv.  Shared memory: K and V (five slabs), three stages of a 64-query
// tile (Q, dO and its aux rows).  Tensor memory: S^T 64 columns, dP^T 64,
// P^T and dS^T 32 each (16-bit), dV 128, dK 192: all 512, which is what holds
// the query tile at 64 (S^T and dP^T then read their first operand from
// shared memory for 64 columns only and are bound by that: about 1600 cycles
// a 128 x 64 tile beside 1280 of arithmetic).
// ---------------------------------------------------------------------------
constexpr uint32_t STAGES = 3;
constexpr uint32_t STAGE = 5 * HSLAB;
constexpr uint32_t K_K = 0, K_V = 3 * SLAB, K_ST = 5 * SLAB, K_AUX = K_ST + STAGES * STAGE,
                   K_BAR = K_AUX + STAGES * 2 * QT * 4;
constexpr uint32_t K_KVFULL = K_BAR, K_FULL = K_KVFULL + 8, K_KDONE = K_FULL + 8 * STAGES, K_SFULL = K_KDONE + 8 * STAGES,
                   K_DPFULL = K_SFULL + 8, K_SREAD = K_DPFULL + 8, K_DPREAD = K_SREAD + 8, K_PFULL = K_DPREAD + 8,
                   K_DSFULL = K_PFULL + 8, K_DRAIN = K_DSFULL + 8,
                   K_TMEM = K_DRAIN + 16, K_FAILED = K_TMEM + 4;
constexpr uint32_t K_SMEM = K_FAILED + 4 + 1024;
static_assert(K_SMEM <= 232448, "shared memory of one CTA");

template <bool FP16>
__global__ void __launch_bounds__(BWD_THREADS, 1)
    latent_dkv_kernel(const __grid_constant__ LatentParams p, const __grid_constant__ BwdMaps maps, int slots) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
    volatile uint32_t* failed = reinterpret_cast<volatile uint32_t*>(smem + K_FAILED);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t limit = p.wait_limit != 0u ? p.wait_limit : WAIT_LIMIT;

    int n, j0;
    LatentSeq s;
    int slot, h;
    latent_order(p, (int)blockIdx.x, slots, false, slot, h);
    const bool found = latent_find(p, p.cu_k, p.Tk, slot, LAT_TILE, n, j0, s);
    const int key0 = found ? j0 * LAT_TILE : 0;
    const bool checks = p.Tq == 0 && blockIdx.x == 0;                   // (elsewhere the launch of the tables does)
    if (!found || key0 >= s.lk) {
        if (checks) check_offsets(p, tid, BWD_THREADS);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const int shift = s.lk - s.lq;
    const int first = p.causal ? max(0, key0 - shift) / QT : 0;         // query tile
    const int steps = max(0, (s.lq + QT - 1) / QT - first);
    const int slot0 = p.cu_q == nullptr ? n * ((p.Tq + QT - 1) / QT) : (int)(s.q0 / QT) + n;

    if (tid == 32) {
        prefetch_map(&maps.kv);
        prefetch_map(&maps.pe);
        prefetch_map(&maps.q64);
        prefetch_map(&maps.dout64);
    }
    if (tid == 0) {
        mbar_init(base + K_KVFULL, 1);
        for (uint32_t i = 0; i < STAGES; ++i) mbar_init(base + K_FULL + 8 * i, 1), mbar_init(base + K_KDONE + 8 * i, 1);
        mbar_init(base + K_SFULL, 1);
        mbar_init(base + K_DPFULL, 1);
        mbar_init(base + K_SREAD, 8);
        mbar_init(base + K_DPREAD, 8);
        mbar_init(base + K_PFULL, 8);
        mbar_init(base + K_DSFULL, 8);
        mbar_init(base + K_DRAIN, 1);
        mbar_init(base + K_DRAIN + 8, 1);
        *failed = 0u;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(base + K_TMEM, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + K_TMEM);
    const uint32_t t_s = tmem, t_dp = tmem + 64, t_p = tmem + 128, t_ds = tmem + 160, t_dv = tmem + 192, t_dk = tmem + 320;

    if (warp == 10) {
        if (lane == 0 && steps > 0) {
            const int tk = (int)s.k0 + key0;
            mbar_arrive_expect_tx(base + K_KVFULL, 5 * SLAB);
            for (uint32_t c = 0; c < 2; ++c) {
                tma_load_3d(base + K_K + c * SLAB, &maps.kv, 64 * c, h, tk, base + K_KVFULL);
                tma_load_3d(base + K_V + c * SLAB, &maps.kv, LAT_N + 64 * c, h, tk, base + K_KVFULL);
            }
            tma_load_3d(base + K_K + 2 * SLAB, &maps.pe, 0, 0, tk, base + K_KVFULL);
            uint32_t i = 0;
            for (; i < (uint32_t)steps; ++i) {
                const uint32_t st = i % STAGES, bar = base + K_FULL + 8 * st, dst = base + K_ST + st * STAGE;
                if (i >= STAGES && !wait_phase(base + K_KDONE + 8 * st, (i / STAGES - 1) & 1, limit, failed)) break;
                const int tile = first + (int)i, tq = (int)s.q0 + tile * QT;
                mbar_arrive_expect_tx(bar, STAGE + 2 * QT * 4);
                for (uint32_t c = 0; c < 3; ++c) tma_load_3d(dst + c * HSLAB, &maps.q64, 64 * c, h, tq, bar);
                for (uint32_t c = 0; c < 2; ++c) tma_load_3d(dst + (3 + c) * HSLAB, &maps.dout64, 64 * c, h, tq, bar);
                bulk_g2s(base + K_AUX + st * 2 * QT * 4, p.aux + ((long long)(slot0 + tile) * p.H + h) * 2 * QT, 2 * QT * 4,
                         bar);
            }
            // every copy issued here has landed before the CTA ends
            mbar_wait(base + K_KVFULL, 0, DRAIN_LIMIT);
            for (uint32_t k = i > STAGES ? i - STAGES : 0; k < i; ++k)
                mbar_wait(base + K_FULL + 8 * (k % STAGES), (k / STAGES) & 1, DRAIN_LIMIT);
        }
    } else if (warp >= 8) {
        const MmaType ty = FP16 ? T_F16 : T_BF16;
        const uint32_t id_s = idesc_f16(ty, 128, QT, false, false), id_v = idesc_f16(ty, 128, 128, false, true),
                       id_k = idesc_f16(ty, 128, 192, false, true);
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = ok && wait_warp(base + bar, parity, limit, failed);
            return ok;
        };
        auto stage = [&](int i) { return base + K_ST + ((uint32_t)i % STAGES) * STAGE; };
        auto score = [&](int i) {
            if (!wait(K_FULL + 8 * (i % STAGES), (i / STAGES) & 1)) return;
            const int past = s.lq - (first + i) * QT;
            if (past < QT) {
                // rows past the sequence's end hold whatever follows: zero weights have to meet zeros
                for (int r = past + (lane >> 3); r < QT; r += 4)
#pragma unroll
                    for (int c = 0; c < 5; ++c)
                        *reinterpret_cast<uint4*>(smem + (stage(i) - base) + c * HSLAB + r * 128 + (lane & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                fence_async_smem();
                __syncwarp();
            }
            const Desc a = desc_k(base + K_K), b = desc_k(stage(i));
#pragma unroll
            for (int ks = 0; ks < 12; ++ks)
                mma_ss(t_s, a + ((ks >> 2) * (SLAB / 16) + (ks & 3) * 2), b + ((ks >> 2) * (HSLAB / 16) + (ks & 3) * 2), id_s,
                       ks > 0);
            mma_commit_warp(base + K_SFULL);
        };
        auto grad_p = [&](int i) {
            const Desc a = desc_k(base + K_V), b = desc_k(stage(i) + 3 * HSLAB);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
                mma_ss(t_dp, a + ((ks >> 2) * (SLAB / 16) + (ks & 3) * 2), b + ((ks >> 2) * (HSLAB / 16) + (ks & 3) * 2), id_s,
                       ks > 0);
            mma_commit_warp(base + K_DPFULL);
        };
        if (warp == 8) {
            if (steps > 0 && wait(K_KVFULL, 0)) {
                score(0);
                if (ok) grad_p(0);
            }
            for (int i = 0; i + 1 < steps && ok; ++i) {
                if (!wait(K_SREAD, i & 1)) break;
                tc_fence_after();
                score(i + 1);
                if (!ok || !wait(K_DPREAD, i & 1)) break;
                tc_fence_after();
                grad_p(i + 1);
            }
        } else {
            for (int i = 0; i < steps && wait(K_PFULL, i & 1); ++i) {
                tc_fence_after();
                const Desc bv = desc_mn(stage(i) + 3 * HSLAB, QT), bk = desc_mn(stage(i), QT);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_ts(t_dv, t_p + 8 * ks, bv + 128 * ks, id_v, i + ks > 0);
                if (!wait(K_DSFULL, i & 1)) break;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_ts(t_dk, t_ds + 8 * ks, bk + 128 * ks, id_k, i + ks > 0);
                mma_commit_warp(base + K_KDONE + 8 * (i % STAGES));
            }
        }
        // every product issued here is done before the tensor memory is freed
        mma_commit_warp(base + K_DRAIN + 8 * (warp & 1));
        mbar_wait(base + K_DRAIN + 8 * (warp & 1), 0, DRAIN_LIMIT);
    } else {
        const int g = warp >> 2, key = key0 + (warp & 3) * 32 + lane;   // queries 32 g .. of a tile
        const uint32_t quad = (uint32_t)(warp & 3) << 21;
        const float c = p.scale * LOG2E;
        const int gs = grad_shift<FP16>(p, s, h);
        const float to_ds = pow2(gs - (int)P_SHIFT<FP16>);
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = ok && wait_warp(base + bar, parity, limit, failed);
            return ok;
        };
        for (int i = 0; i < steps; ++i) {
            const uint32_t st = (uint32_t)i % STAGES;
            if (!wait(K_FULL + 8 * st, (i / STAGES) & 1) || !wait(K_SFULL, i & 1)) break;
            tc_fence_after();
            const float4* aux = reinterpret_cast<const float4*>(smem + K_AUX + st * 2 * QT * 4) + 8 * g;
            float x[32];
            tmem_ld32(t_s + 32 * g + quad, x);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(base + K_SREAD);
            // query e of these 32 sees this key iff e >= lo
            const int lo = p.causal ? key - shift - (first + i) * QT - 32 * g : 0;
            const bool cut = __any_sync(0xffffffffu, lo > 0);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                const float4 l = aux[e >> 2];
                x[e] = ex2(fmaf(x[e], c, -l.x));
                x[e + 1] = ex2(fmaf(x[e + 1], c, -l.y));
                x[e + 2] = ex2(fmaf(x[e + 2], c, -l.z));
                x[e + 3] = ex2(fmaf(x[e + 3], c, -l.w));
            }
            if (cut) {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = e >= lo ? x[e] : 0.f;
            }
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) w[e >> 1] = pack2<FP16>(x[e], x[e + 1]);
            // P and dS are free once the step before is done
            if (i > 0 && !wait(K_KDONE + 8 * ((i - 1) % STAGES), ((i - 1) / STAGES) & 1)) break;
            tc_fence_after();
            tmem_st16(t_p + 16 * g + quad, w);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(base + K_PFULL);
            if (!wait(K_DPFULL, i & 1)) break;
            tc_fence_after();
            float d[32];
            tmem_ld32(t_dp + 32 * g + quad, d);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(base + K_DPREAD);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                const float4 l = aux[2 * QT / 8 + (e >> 2)];
                d[e] = x[e] * (d[e] - l.x);
                d[e + 1] = x[e + 1] * (d[e + 1] - l.y);
                d[e + 2] = x[e + 2] * (d[e + 2] - l.z);
                d[e + 3] = x[e + 3] * (d[e + 3] - l.w);
            }
            if constexpr (FP16) {
#pragma unroll
                for (int e = 0; e < 32; ++e) d[e] *= to_ds;            // P's factor off, dS's on
            }
            if (cut) {
#pragma unroll
                for (int e = 0; e < 32; ++e) d[e] = e >= lo ? d[e] : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 32; e += 2) w[e >> 1] = pack2<FP16>(d[e], d[e + 1]);
            tmem_st16(t_ds + 16 * g + quad, w);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(base + K_DSFULL);
        }
        if (steps > 0 && ok) wait(K_KDONE + 8 * ((steps - 1) % STAGES), ((steps - 1) / STAGES) & 1);
        if (bar_and_named(1, 256, ok)) {
            // every product is done: K's and V's slabs take dk and dv, the stages the shared key's part in 32 bits
            tc_fence_after();
            const int r = key - key0;
            const float f = g == 0 ? 1.f : p.scale, undo = pow2(g == 0 ? -(int)P_SHIFT<FP16> : -gs);
            const uint32_t src = (g == 0 ? t_dv : t_dk) + quad;
#pragma unroll 1
            for (int b = 0; b < (g == 0 ? 4 : 6); ++b) {
                float d[32];
                if (steps > 0) {
                    tmem_ld32(src + 32 * b, d);
                    tmem_ld_wait();
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) d[e] = steps > 0 ? (FP16 ? d[e] * undo : d[e]) * f : 0.f;
                if (b < 4) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        *reinterpret_cast<uint4*>(staged(smem + K_K, r, (g == 0 ? 16 : 0) + 4 * b + (e >> 3))) =
                            make_uint4(pack2<FP16>(d[e], d[e + 1]), pack2<FP16>(d[e + 2], d[e + 3]),
                                       pack2<FP16>(d[e + 4], d[e + 5]), pack2<FP16>(d[e + 6], d[e + 7]));
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4*>(staged(smem + K_ST, r, 8 * (b - 4) + (e >> 2))) =
                            make_float4(d[e], d[e + 1], d[e + 2], d[e + 3]);
                }
            }
            bar_and_named(1, 256, true);
            const long long rows = p.cu_k != nullptr ? p.Tk : (long long)p.N * p.Tk;
            const int count = min(LAT_TILE, s.lk - key0);
            copy_rows<LAT_KV / 8>(smem + K_K, static_cast<uint16_t*>(p.dkv) + ((s.k0 + key0) * p.H + h) * LAT_KV,
                                  (long long)p.H * LAT_KV * 2, count, tid, 256);
            copy_rows<LAT_P / 4>(smem + K_ST, p.dpe_part + (h * rows + s.k0 + key0) * LAT_P, LAT_P * 4, count, tid, 256);
        }
    }
    tc_fence_before();
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");   // what follows this launch also follows the dq kernel
    if (warp == 8) tmem_dealloc(tmem, 512);
    if (checks) check_offsets(p, tid, BWD_THREADS);
    if (tid == 0 && *failed) set_status(p.status, STATUS_TIMEOUT);
}

template <bool FP16>
__global__ void __launch_bounds__(256) latent_dpe_kernel(const __grid_constant__ LatentParams p, long long quads) {
    const long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (e >= quads) return;
    const float4* part = reinterpret_cast<const float4*>(p.dpe_part) + e;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int h = 0; h < p.H; ++h) {
        const float4 v = part[h * quads];
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
    }
    static_cast<uint2*>(p.dk_pe)[e] = make_uint2(pack2<FP16>(sum.x, sum.y), pack2<FP16>(sum.z, sum.w));
}

template <bool FP16>
cudaError_t launch(const LatentParams& p, const BwdMaps& maps, cudaStream_t stream) {
    const bool varlen = p.cu_q != nullptr;
    cudaError_t e = cudaFuncSetAttribute(latent_dq_kernel<FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)D_SMEM);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(latent_dkv_kernel<FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)K_SMEM);
    if (e != cudaSuccess) return e;
    // The dq and key kernels may be set up, and begin, beside the end of the launch before them (see there).
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(BWD_THREADS);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p.Tq > 0) {
        const int aux_slots = latent_slots(varlen, p.Tq, p.N, QT);
        const bool sizes = FP16 && p.Tk > 0;
        if (sizes) {   // the maxima of grad_sizes begin at zero
            const size_t rows = varlen ? p.Tk : (size_t)p.N * p.Tk;
            e = cudaMemsetAsync(p.dk_pe, 0, rows * LAT_P * 2, stream);
            if (e != cudaSuccess) return e;
        }
        latent_aux_kernel<FP16><<<dim3(aux_slots + (sizes ? latent_slots(varlen, p.Tk, p.N, QT) : 0), p.H), 256, 0, stream>>>(
            p, aux_slots);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        const int slots = latent_slots(varlen, p.Tq, p.N, LAT_TILE);
        cfg.gridDim = dim3((unsigned)(slots * p.H));
        cfg.dynamicSmemBytes = D_SMEM;
        e = cudaLaunchKernelEx(&cfg, latent_dq_kernel<FP16>, p, maps, slots);
        if (e != cudaSuccess) return e;
    }
    if (p.Tk > 0) {
        const int slots = latent_slots(varlen, p.Tk, p.N, LAT_TILE);
        cfg.gridDim = dim3((unsigned)(slots * p.H));
        cfg.dynamicSmemBytes = K_SMEM;
        cfg.numAttrs = p.Tq > 0 ? 1 : 0;
        e = cudaLaunchKernelEx(&cfg, latent_dkv_kernel<FP16>, p, maps, slots);
        if (e != cudaSuccess) return e;
        const long long quads = (varlen ? p.Tk : (long long)p.N * p.Tk) * (LAT_P / 4);
        latent_dpe_kernel<FP16><<<(unsigned)((quads + 255) / 256), 256, 0, stream>>>(p, quads);
    }
    return cudaGetLastError();
}

}  // namespace

// Floats of the tables that latent_aux_kernel writes.
unsigned long long latent_aux_floats(int B, int Tq, int H, int N) {
    const int varlen = latent_slots(true, Tq, N, QT), fixed = latent_slots(false, Tq, B, QT);
    return (unsigned long long)(varlen > fixed ? varlen : fixed) * H * 2ull * QT;
}

cudaError_t launch_latent_bwd(const LatentParams& p, bool fp16, cudaStream_t stream) {
    const bool varlen = p.cu_q != nullptr;
    const long long rows_q = varlen ? p.Tq : (long long)p.N * p.Tq, rows_k = varlen ? p.Tk : (long long)p.N * p.Tk;
    // without rows on one side nothing is loaded from it: any valid tensor does
    const void* any = rows_q > 0 ? p.q : p.kv;
    if (rows_q == 0 && rows_k == 0) return cudaSuccess;
    const void* q = rows_q > 0 ? p.q : any;
    const void* dout = rows_q > 0 ? p.dout : any;
    const void* kv = rows_k > 0 ? p.kv : any;
    const void* pe = rows_k > 0 ? p.k_pe : any;
    const long long tq = rows_q > 0 ? rows_q : 1, tk = rows_k > 0 ? rows_k : 1;
    BwdMaps maps;
    if (!latent_row_map(&maps.q, q, LAT_QK, p.H, tq, (long long)p.H * LAT_QK, LAT_TILE) ||
        !latent_row_map(&maps.dout, dout, LAT_V, p.H, tq, (long long)p.H * LAT_V, LAT_TILE) ||
        !latent_row_map(&maps.kv, kv, LAT_KV, p.H, tk, (long long)p.H * LAT_KV, LAT_TILE) ||
        !latent_row_map(&maps.pe, pe, LAT_P, 1, tk, p.k_pe_stride, LAT_TILE) ||
        !latent_row_map(&maps.q64, q, LAT_QK, p.H, tq, (long long)p.H * LAT_QK, QT) ||
        !latent_row_map(&maps.dout64, dout, LAT_V, p.H, tq, (long long)p.H * LAT_V, QT))
        return cudaErrorInvalidValue;
    return fp16 ? launch<true>(p, maps, stream) : launch<false>(p, maps, stream);
}

}  // namespace kda
