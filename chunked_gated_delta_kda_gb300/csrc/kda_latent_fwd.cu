// Expanded latent attention, forward.
//
// One pass over the keys with the softmax's running maximum m and sum l:
//   S = Q K^T (tcgen05, 192 channels: 128 of the head, 64 shared), P = exp2(c S - c m), O = O + P V,
// with c = scale log2(e).  m is a reference, not the exact maximum: it follows
// the row maximum only when that has grown by more than 2^8 in P's terms, so
// that O is rarely rescaled; P stays below 2^8 and the result is the same in
// exact arithmetic.
//
// A CTA owns 256 queries of one head as two tiles of 128 rows, so that one
// tile's softmax runs while the tensor cores work on the other:
//   warps 0-3, 4-7  softmax of tile 0 / 1, one thread a row, and its output
//   warp 8          issues the products
//   warp 9          loads: Q once, then K and V tiles of 128 keys through a
//                   ring of eight 16 KiB slabs (64 columns x 128 rows, as
//                   the tensor map's 128-byte swizzle stores them)
// Tensor memory: S (128 columns) and O (128) of both tiles; P, as 16-bit
// operand of the second product, takes the first half of its S columns.  The
// products of one tile are issued in the order P V (j), Q K^T (j + 1); the
// tensor pipe keeps that order, so S may overwrite P, and a full S means that
// the P V before it is done.
//
// P is rounded to the tensors' type as an operand of the second product (32-bit
// operands run at half the rate and twice the columns): bf16 o is off by 0.0020
// of its norm, 0.0015 of that its own rounding (B=4 T=8192).
//
// B=4 T=8192 H=16 causal: 0.82 ms in a few calls after a pause, 1670 TFLOP/s of
// the mask's pairs, and 0.90, 1530, once calls back to back have brought the GPU
// to its power limit (a library product then runs at 1710); T=8192 H=8 0.116 ms
// in either state, 1480.  A step of both tiles is 2560 cycles of products and takes
// 3460: a tile's softmax (1500 cycles from its scores to its weights) and its
// two products follow each other, and the other tile fills the gap but for
// that.  Short sequences are bound by a CTA's first loads and last stores,
// which only other CTAs' work could cover.  Not better: the weights handed over
// in two halves (T=8192 H=8 127 us), a warp of its own for each tile's products
// (140), the output staged in shared memory as the backward's is (no change).
#include "kda_latent_mma.cuh"

#include <cudaTypedefs.h>

namespace kda {

PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder();

bool latent_row_map(CUtensorMap* m, const void* base, int width, int heads, long long tokens, long long row_stride,
                    int box_rows) {
    const PFN_cuTensorMapEncodeTiled_v12000 fn = tmap_encoder();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)width * 2u, (cuuint64_t)row_stride * 2u};
    const cuuint32_t box[3] = {64u, 1u, (cuuint32_t)box_rows};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

constexpr int FWD_ROWS = 2 * LAT_TILE;
constexpr int FWD_THREADS = 384;                        // warps 10 and 11 hold registers for the softmax (and check offsets)
constexpr uint32_t SLAB = 64 * LAT_TILE * 2;            // 16 KiB
constexpr uint32_t RING = 8;
constexpr uint32_t F_Q = 0;                             // [tile][3 slabs]
constexpr uint32_t F_RING = 6 * SLAB;
constexpr uint32_t F_BAR = F_RING + RING * SLAB;
constexpr uint32_t F_KFULL = F_BAR;                     // [2] K of steps j & 1
constexpr uint32_t F_VFULL = F_KFULL + 16;              // [2]
constexpr uint32_t F_VEMPTY = F_VFULL + 16;             // [2]
constexpr uint32_t F_QFULL = F_VEMPTY + 16;             // [2]
constexpr uint32_t F_SFULL = F_QFULL + 16;              // [tile][step & 1]
constexpr uint32_t F_PFULL = F_SFULL + 32;              // [2]
constexpr uint32_t F_ODONE = F_PFULL + 16;              // [2]
constexpr uint32_t F_DRAIN = F_ODONE + 16;
constexpr uint32_t F_TMEM = F_DRAIN + 8;
constexpr uint32_t F_FAILED = F_TMEM + 4;
constexpr uint32_t F_BYTES = F_FAILED + 4;
constexpr uint32_t F_SMEM = F_BYTES + 1024;             // room to align the base
static_assert(F_SMEM <= 232448, "shared memory of one CTA");

constexpr float RESCALE_LOG2 = 8.f;

struct FwdMaps {
    CUtensorMap q, kv, pe;
};

// Where a part's row keeps its 16-byte piece: swizzled, so that a thread a row
// (written) and a warp a row (read) both spread over the banks.
__device__ __forceinline__ uint32_t part_at(uint32_t row, uint32_t piece) {
    return F_RING + row * 512u + ((piece ^ (row & 31u)) * 16u);
}

// ---- tile pairs whose keys several CTAs share, chosen on the device ----
// A pair's keys are walked by one CTA, so where one sequence has many more
// keys than the others (a chunk behind a long prefix beside short prompts) its
// pairs end last by far.  A first kernel counts each pair's key tiles, gives
// those that are long against an SM's share of all of them up to 16 CTAs, and
// sorts the work; the parts (O, m and l in 32 bits) are joined by a third.  The
// two cost some 5 us where nothing is shared.  Without / with, in us, H=16:
// queries 512, 129, 1, 1000 on 8192, 4039, 3000, 1000 keys 121 / 67; 64, 64, 2048
// on 512, 16384, 2048 191 / 64; H=8: 14 x 1, 1, 1 on 14 x 500, 9000, 30000 338 /
// 59; 6 x 300 on 500 to 8000 114 / 48; 4 x 2048 on themselves 54 / 48 (from the
// order); H=4: 30 x 1 on 3000 each 47 / 53.  Clusters with ranks that leave where
// a pair is short hold their SMs to the end of the cluster: 2 x 4096, 8 heads
// 116 -> 298.
constexpr int SHARE_SLOTS = 512;       // tile pairs of a head, at most
constexpr int SHARE_PARTS = 256;       // parts of 256 rows, over all heads
constexpr int SHARE_RANKS = 16;        // CTAs of a pair, at most
constexpr int SHARE_STEPS = 16;        // key tiles below which a pair is not shared
constexpr float SHARE_LEAST = 8.f;     // key tiles that are worth a part
constexpr long long SHARE_FLOATS = FWD_ROWS * (LAT_V + 2);   // of a part: O as [32][256 rows][4], m and l of each row
// Records: an item a CTA and head (x: slot or -1, y: rank, z: ranks, w: first part); behind the items an entry a shared
// pair (x: first row, y: rows or -1, z, w as before).
__host__ __device__ __forceinline__ int share_items(int slots, int H) { return slots + SHARE_PARTS / H; }
static_assert(SHARE_SLOTS + SHARE_PARTS + SHARE_PARTS / 2 <= LATENT_SHARE_ITEMS, "records");
__host__ __device__ __forceinline__ int share_pairs(int H) { return SHARE_PARTS / (2 * H); }

// Key tiles of a tile pair's two query tiles.
__device__ __forceinline__ void pair_tiles(const LatentParams& p, const LatentSeq& s, int row0, int (&nt)[2]) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int first = row0 + t * LAT_TILE, last = min(first + LAT_TILE, s.lq) - 1;
        const int kmax = first >= s.lq ? 0 : p.causal ? min(s.lk, last + s.lk - s.lq + 1) : s.lk;
        nt[t] = kmax > 0 ? (kmax + LAT_TILE - 1) / LAT_TILE : 0;
    }
}

__global__ void __launch_bounds__(SHARE_SLOTS) latent_share_kernel(const __grid_constant__ LatentParams p, int slots) {
    __shared__ int keys[SHARE_SLOTS], counts[SHARE_SLOTS], sums[SHARE_SLOTS / 32], cu[SHARE_SLOTS + 1];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int items = share_items(slots, p.H), pairs = share_pairs(p.H);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (t < WS_CLEAR / 4) p.status[t] = 0u;
    for (int i = t; i < items + pairs; i += SHARE_SLOTS) p.share_items[i] = make_int4(-1, -1, 0, 0);
    for (int i = t; i <= p.N; i += SHARE_SLOTS) cu[i] = p.cu_q[i];
    __syncthreads();
    check_offsets(p, t, SHARE_SLOTS);
    int n, j, steps = -1;              // -1: no such pair
    LatentSeq s;
    if (t < slots) {
        latent_slot(cu, p.Tq, p.N, t, FWD_ROWS, n, j);
        if (latent_seq(p, n, s) && (long long)j * FWD_ROWS < s.lq) {
            int nt[2];
            pair_tiles(p, s, j * FWD_ROWS, nt);
            steps = max(nt[0], nt[1]);
        }
    }
    const int mine = __reduce_add_sync(0xffffffffu, max(steps, 0));
    if (lane == 0) sums[warp] = mine;
    __syncthreads();
    int total = 0;
    for (int w = 0; w < SHARE_SLOTS / 32; ++w) total += sums[w];
    // an SM's share of the key tiles of all heads, and the CTAs that bring a pair's nearest to it
    const float share = fmaxf((float)total * (float)p.H * (1.f / 152.f), SHARE_LEAST);
    int ranks = steps < SHARE_STEPS ? 1 : max(1, min(SHARE_RANKS, (int)((float)steps / share + 0.5f)));
    // where a shared pair's parts and its entry go
    int parts = ranks > 1 ? ranks : 0, x = parts | (parts > 0 ? 1 << 16 : 0);
    const int own = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    for (int w = 0; w < warp; ++w) x += sums[w];
    x -= own;
    const int base = x & 0xffff, entry = x >> 16;
    if (parts > 0 && ((base + parts) * p.H > SHARE_PARTS || entry >= pairs)) ranks = 1, parts = 0;
    const int each = steps < 0 ? -1 : (steps + ranks - 1) / ranks;   // what orders the work: the longest first
    keys[t] = each;
    counts[t] = steps < 0 ? 0 : ranks;
    __syncthreads();
    if (steps < 0) return;
    int at = 0;
    for (int u = 0; u < slots; ++u)
        if (keys[u] > each || (keys[u] == each && u < t)) at += counts[u];
    for (int k = 0; k < ranks; ++k) p.share_items[at + k] = make_int4(t, k, ranks, base);
    if (parts > 0)
        p.share_items[items + entry] = make_int4((int)s.q0 + j * FWD_ROWS, min(FWD_ROWS, s.lq - j * FWD_ROWS), ranks, base);
}

// Eight CTAs a shared pair and head, 16 channels each, a thread a row.
template <bool FP16>
__global__ void __launch_bounds__(FWD_ROWS) latent_share_join_kernel(const __grid_constant__ LatentParams p, int slots) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int h = blockIdx.x % p.H, r = threadIdx.x;
    const int4 it = p.share_items[share_items(slots, p.H) + blockIdx.x / p.H];
    if (r >= it.y) return;
    const float c = p.scale * 1.4426950408889634f;
    auto part = [&](int k) { return p.share_parts + ((long long)(it.w + k) * p.H + h) * SHARE_FLOATS; };
    float m = -INFINITY, l = 0.f, o[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = 0.f;
    auto stat = [&](int k) { return reinterpret_cast<const float2*>(part(k) + FWD_ROWS * LAT_V)[r]; };
#pragma unroll 4
    for (int k = 0; k < it.z; ++k) m = fmaxf(m, stat(k).x);
#pragma unroll 4
    for (int k = 0; k < it.z; ++k) {
        const float2 st = stat(k);
        const float f = st.x == -INFINITY ? 0.f : ex2((st.x - m) * c);
        l += f * st.y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 v = reinterpret_cast<const float4*>(part(k))[(4 * blockIdx.y + e) * FWD_ROWS + r];
            o[4 * e] += f * v.x;
            o[4 * e + 1] += f * v.y;
            o[4 * e + 2] += f * v.z;
            o[4 * e + 3] += f * v.w;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const long long at = ((long long)it.x + r) * p.H + h;
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = pack2<FP16>(o[2 * e] * inv, o[2 * e + 1] * inv);
    uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o_out) + at * LAT_V + 16 * blockIdx.y);
    out[0] = make_uint4(w[0], w[1], w[2], w[3]);
    out[1] = make_uint4(w[4], w[5], w[6], w[7]);
    if (blockIdx.y == 0 && p.lse_out) p.lse_out[at] = l == 0.f ? -INFINITY : m * p.scale + logf(l);
}

enum Split { WHOLE, CLUSTER, SHARED };

// CLUSTER: the CTAs of a cluster share the keys of a tile pair, each with its
// own m, l and O, and join them through the cluster's shared memory.  SHARED:
// see above.
template <bool FP16, int SPLIT>
__global__ void __launch_bounds__(FWD_THREADS, 1)
    latent_fwd_kernel(const __grid_constant__ LatentParams p, const __grid_constant__ FwdMaps maps, int slots) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
    volatile uint32_t* failed = reinterpret_cast<volatile uint32_t*>(smem + F_FAILED);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t limit = p.wait_limit != 0u ? p.wait_limit : WAIT_LIMIT;

    int n, j0;
    LatentSeq s;
    int slot, h;
    int4 item = make_int4(0, 0, 1, 0);
    if constexpr (SPLIT == SHARED) {
        // only the records are waited for: the tensors were there before the kernel that writes them began
        asm volatile("griddepcontrol.wait;");
        const volatile int* at = reinterpret_cast<const volatile int*>(p.share_items + blockIdx.x / p.H);
        item = make_int4(at[0], at[1], at[2], at[3]);
        slot = item.x;
        h = blockIdx.x % p.H;
        if (slot < 0) return;
    } else {
        latent_order(p, (int)(SPLIT == CLUSTER ? blockIdx.x / cluster_size() : blockIdx.x), slots, true, slot, h);
    }
    const bool found = latent_find(p, p.cu_q, p.Tq, slot, FWD_ROWS, n, j0, s);
    const int row0 = found ? j0 * FWD_ROWS : 0;
    const bool checks = SPLIT != SHARED && blockIdx.x == 0;
    if (!found || row0 >= s.lq) {         // all CTAs of a cluster alike
        if (checks) check_offsets(p, tid, FWD_THREADS);
        return;
    }
    const int shift = s.lk - s.lq;
    int nt[2];   // key tiles that each query tile needs
    pair_tiles(p, s, row0, nt);
    int j_first = 0;   // first key tile of this CTA
    if constexpr (SPLIT != WHOLE) {
        const int ranks = SPLIT == CLUSTER ? (int)cluster_size() : item.z, rank = SPLIT == CLUSTER ? (int)cluster_rank() : item.y;
        const int all = max(nt[0], nt[1]), each = (all + ranks - 1) / ranks;
        j_first = min(all, rank * each);
        for (int t = 0; t < 2; ++t) nt[t] = max(0, min(nt[t] - j_first, each));
    }
    const int steps = max(nt[0], nt[1]);

    if (tid == 32) {
        prefetch_map(&maps.q);
        prefetch_map(&maps.kv);
        prefetch_map(&maps.pe);
    }
    if (tid == 0) {
        for (uint32_t t = 0; t < 2; ++t) {
            mbar_init(base + F_KFULL + 8 * t, 1);
            mbar_init(base + F_VFULL + 8 * t, 1);
            mbar_init(base + F_VEMPTY + 8 * t, 1);
            mbar_init(base + F_QFULL + 8 * t, 1);
            mbar_init(base + F_SFULL + 16 * t, 1);
            mbar_init(base + F_SFULL + 16 * t + 8, 1);
            mbar_init(base + F_PFULL + 8 * t, 4);
            mbar_init(base + F_ODONE + 8 * t, 1);
        }
        mbar_init(base + F_DRAIN, 1);
        *failed = 0u;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(base + F_TMEM, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + F_TMEM);
    // slab sequence: K of step j at 5 j .. 5 j + 2, its V at 5 j + 3, 5 j + 4
    auto slab = [&](uint32_t i) { return base + F_RING + (i % RING) * SLAB; };

    if (warp >= 8) {
        // 168 registers a thread at launch: the softmax's 256 threads take 208, these 88 (2 x 208 + 88 = 3 x 168)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 9 && lane == 0 && steps > 0) {
            for (int t = 0; t < 2; ++t) {
                if (nt[t] == 0) continue;
                mbar_arrive_expect_tx(base + F_QFULL + 8 * t, 3 * SLAB);
                for (uint32_t c = 0; c < 3; ++c)
                    tma_load_3d(base + F_Q + (3 * t + c) * SLAB, &maps.q, 64 * c, h, (int)s.q0 + row0 + t * LAT_TILE,
                                base + F_QFULL + 8 * t);
            }
            // Slab i takes the place of slab i - 8: K of step j that of K's last and V's slabs of step j - 2, V of
            // step j that of K's first two of step j - 1, which the last product of S (j - 1) frees.
            const uint32_t s_last = base + F_SFULL + (nt[1] > 0 ? 16 : 0);
            int j = 0;
            bool half = false;   // given up between a step's K and its V
            for (; j < steps; ++j) {
                const int tok = (int)s.k0 + (j_first + j) * LAT_TILE, st = j & 1;
                if (j >= 2 && !wait_phase(base + F_VEMPTY + 8 * st, (j / 2 - 1) & 1, limit, failed)) break;
                mbar_arrive_expect_tx(base + F_KFULL + 8 * st, 3 * SLAB);
                for (int c = 0; c < 2; ++c) tma_load_3d(slab(5 * j + c), &maps.kv, 64 * c, h, tok, base + F_KFULL + 8 * st);
                tma_load_3d(slab(5 * j + 2), &maps.pe, 0, 0, tok, base + F_KFULL + 8 * st);
                if (j >= 1 && !wait_phase(s_last + 8 * ((j - 1) & 1), ((j - 1) >> 1) & 1, limit, failed)) {
                    half = true;
                    break;
                }
                mbar_arrive_expect_tx(base + F_VFULL + 8 * st, 2 * SLAB);
                for (int c = 0; c < 2; ++c)
                    tma_load_3d(slab(5 * j + 3 + c), &maps.kv, LAT_N + 64 * c, h, tok, base + F_VFULL + 8 * st);
            }
            // every copy issued here has landed before the CTA ends
            for (int t = 0; t < 2; ++t)
                if (nt[t] > 0) mbar_wait(base + F_QFULL + 8 * t, 0, DRAIN_LIMIT);
            // (given up halfway, step j - 2's have, and its barrier counts step j's)
            for (int k = max(0, half ? j - 1 : j - 2); k < j; ++k) {
                mbar_wait(base + F_KFULL + 8 * (k & 1), (k / 2) & 1, DRAIN_LIMIT);
                mbar_wait(base + F_VFULL + 8 * (k & 1), (k / 2) & 1, DRAIN_LIMIT);
            }
            if (half) mbar_wait(base + F_KFULL + 8 * (j & 1), (j / 2) & 1, DRAIN_LIMIT);
        } else if (warp == 8) {
            const uint32_t id = idesc_f16(FP16 ? T_F16 : T_BF16, 128, 128, false, false);
            const uint32_t idv = idesc_f16(FP16 ? T_F16 : T_BF16, 128, 128, false, true);
            const uint32_t idv64 = idesc_f16(FP16 ? T_F16 : T_BF16, 128, 64, false, true);
            bool ok = true;
            auto wait = [&](uint32_t bar, uint32_t parity) {
                ok = ok && wait_warp(base + bar, parity, limit, failed);
                return ok;
            };
            auto qk = [&](int t, int j, bool loaded) {   // S_t = Q_t K_j^T
                if (!loaded && !wait(F_KFULL + 8 * (j & 1), (j >> 1) & 1)) return;
#pragma unroll
                for (int c = 0; c < 3; ++c) {
                    const Desc a = desc_k(base + F_Q + (3 * t + c) * SLAB), b = desc_k(slab(5 * j + c));
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) mma_ss(tmem + 256 * t, a + 2 * ks, b + 2 * ks, id, c + ks > 0);
                }
                mma_commit_warp(base + F_SFULL + 16 * t + 8 * (j & 1));
            };
            for (int t = 0; t < 2 && ok; ++t)
                if (nt[t] > 0 && wait(F_QFULL + 8 * t, 0)) qk(t, 0, t == 1 && nt[0] > 0);
            for (int j = 0; j < steps && ok; ++j) {
                const uint32_t v = 5 * j + 3;
                if (!wait(F_VFULL + 8 * (j & 1), (j >> 1) & 1)) break;
                if ((j_first + j + 1) * LAT_TILE > s.lk) {
                    // rows past the sequence's end hold whatever follows: zero weights must meet zeros
                    for (int r = s.lk - (j_first + j) * LAT_TILE; r < LAT_TILE; ++r)
                        if (lane < 16)
                            *reinterpret_cast<uint4*>(smem + (slab(v + (lane >> 3)) - base) + r * 128 + (lane & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                    fence_async_smem();
                    __syncwarp();
                }
                bool loaded = false;   // K of the next step
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (j < nt[t]) {
                        if (!wait(F_PFULL + 8 * t, j & 1)) break;
                        tc_fence_after();
                        // O_t += P_t V_j; where the ring wraps between V's two slabs, one product for each
                        const uint32_t d = tmem + 256 * t + 128, a = tmem + 256 * t;
                        const Desc b = desc_mn(slab(v), LAT_TILE);
                        if ((v + 1) % RING != 0) {
#pragma unroll
                            for (int ks = 0; ks < 8; ++ks) mma_ts(d, a + 8 * ks, b + 128 * ks, idv, j + ks > 0);
                        } else {
                            const Desc b1 = desc_mn(slab(v + 1), LAT_TILE);
#pragma unroll
                            for (int ks = 0; ks < 8; ++ks) {
                                mma_ts(d, a + 8 * ks, b + 128 * ks, idv64, j + ks > 0);
                                mma_ts(d + 64, a + 8 * ks, b1 + 128 * ks, idv64, j + ks > 0);
                            }
                        }
                        if (j == nt[t] - 1) mma_commit_warp(base + F_ODONE + 8 * t);
                    }
                    if (t == 1) mma_commit_warp(base + F_VEMPTY + 8 * (j & 1));
                    if (j + 1 < nt[t]) {
                        qk(t, j + 1, loaded);
                        loaded = true;
                    }
                    if (!ok) break;
                }
            }
            // every product issued here is done before the tensor memory is freed
            mma_commit_warp(base + F_DRAIN);
            mbar_wait(base + F_DRAIN, 0, DRAIN_LIMIT);
        } else if (warp >= 10 && checks) {
            check_offsets(p, tid - 320, FWD_THREADS - 320);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int t = warp >> 2;
        const int row = row0 + t * LAT_TILE + (warp & 3) * 32 + lane;
        const uint32_t ts = tmem + 256 * t + ((uint32_t)(warp & 3) << 21);   // this warp's lanes
        const float c = p.scale * 1.4426950408889634f;
        const int kmax = p.causal ? min(s.lk, row + shift + 1) : s.lk;      // keys [0, kmax) count
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = 0; j < nt[t]; ++j) {
            ok = wait_warp(base + F_SFULL + 16 * t + 8 * (j & 1), (j >> 1) & 1, limit, failed);
            if (!ok) break;
            tc_fence_after();
            float x[4][32];
#pragma unroll
            for (int b = 0; b < 4; ++b) tmem_ld32(ts + 32 * b, x[b]);
            tmem_ld_wait();
            const int lim = kmax - (j_first + j) * LAT_TILE;
            if (__any_sync(0xffffffffu, lim < LAT_TILE)) {
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[b][e] = 32 * b + e < lim ? x[b][e] : -INFINITY;
            }
            const float top = fmaxf(fmaxf(max32(x[0]), max32(x[1])), fmaxf(max32(x[2]), max32(x[3])));
            const bool grown = top * c > m * c + RESCALE_LOG2 || (m == -INFINITY && top > m);
            if (__any_sync(0xffffffffu, grown)) {
                const float mn = grown ? top : m;
                const float f = grown ? ex2((m - mn) * c) : 1.f;   // 0 from -inf
                l *= f;
                if (j > 0) {
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        float o[32];
                        tmem_ld32(ts + 128 + 32 * b, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= f;
                        tmem_st32(ts + 128 + 32 * b, o);
                    }
                }
                m = mn;
            }
            const float mc = m == -INFINITY ? 0.f : m * c;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int b = 0; b < 4; b += 2) {
                float w[32];
#pragma unroll
                for (int e = 0; e < 64; e += 2) {
                    float u = x[b + (e >> 5)][e & 31], v = x[b + (e >> 5)][(e & 31) + 1];
                    fma2(u, v, c, -mc);
                    u = ex2(u);
                    v = ex2(v);
                    add2(sum[e & 2], sum[(e & 2) + 1], u, v);
                    w[e >> 1] = __uint_as_float(pack2<FP16>(u, v));
                }
                tmem_st32(ts + 16 * b, w);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(base + F_PFULL + 8 * t);
        }
        if (SPLIT == SHARED && item.z > 1) {
            if (nt[t] > 0 && ok) ok = wait_warp(base + F_ODONE + 8 * t, 0, limit, failed);
            if (ok) {
                tc_fence_after();
                float* part = p.share_parts + ((long long)(item.w + item.y) * p.H + h) * SHARE_FLOATS;
                const int r = t * LAT_TILE + (warp & 3) * 32 + lane;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    float o[32];
                    if (nt[t] > 0) {
                        tmem_ld32(ts + 128 + 32 * b, o);
                        tmem_ld_wait();
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        reinterpret_cast<float4*>(part)[(8 * b + (e >> 2)) * FWD_ROWS + r] =
                            nt[t] > 0 ? make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                reinterpret_cast<float2*>(part + FWD_ROWS * LAT_V)[r] = make_float2(m, l);
            }
        } else if constexpr (SPLIT != CLUSTER) {
            if (nt[t] > 0 && ok) ok = wait_warp(base + F_ODONE + 8 * t, 0, limit, failed);
            if (ok) {
                tc_fence_after();
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const long long at = (s.q0 + row) * p.H + h;
                uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o_out) + at * LAT_V);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    float o[32];
                    if (nt[t] > 0) {
                        tmem_ld32(ts + 128 + 32 * b, o);
                        tmem_ld_wait();
                    }
                    if (row < s.lq) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint32_t r[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                r[k] = l == 0.f ? 0u : pack2<FP16>(o[e + 2 * k] * inv, o[e + 2 * k + 1] * inv);
                            out[4 * b + (e >> 3)] = make_uint4(r[0], r[1], r[2], r[3]);
                        }
                    }
                }
                if (row < s.lq && p.lse_out) p.lse_out[at] = l == 0.f ? -INFINITY : m * p.scale + logf(l);
            }
        } else {
            // the ring is free once both tiles' products are done; it takes this CTA's part of all 256 rows
            for (int k = 0; k < 2; ++k)
                if (nt[k] > 0 && ok) ok = wait_warp(base + F_ODONE + 8 * k, 0, limit, failed);
            if (ok) {
                tc_fence_after();
                const int r = t * LAT_TILE + (warp & 3) * 32 + lane;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    float o[32];
                    if (nt[t] > 0) {
                        tmem_ld32(ts + 128 + 32 * b, o);
                        tmem_ld_wait();
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4*>(smem + part_at(r, 8 * b + (e >> 2))) =
                            nt[t] > 0 ? make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                reinterpret_cast<float2*>(smem + F_Q)[r] = make_float2(m, l);
            }
        }
    }
    if constexpr (SPLIT == CLUSTER) {
        // every CTA of the cluster, failed or not, passes both barriers: the parts are written; they are read
        __syncwarp();
        cluster_barrier();
        if (warp < 8) {
            const uint32_t ranks = cluster_size(), share = FWD_ROWS / ranks;
            const float c = p.scale * 1.4426950408889634f;
            for (uint32_t r = cluster_rank() * share + warp; r < (cluster_rank() + 1) * share; r += 8) {
                const int row = row0 + (int)r;
                if (row >= s.lq) break;
                float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
                for (uint32_t k = 0; k < ranks; ++k)
                    m = fmaxf(m, ld_cluster2(cluster_addr(base + F_Q + 8 * r, k)).x);
                for (uint32_t k = 0; k < ranks; ++k) {
                    const float2 st = ld_cluster2(cluster_addr(base + F_Q + 8 * r, k));
                    const float f = st.x == -INFINITY ? 0.f : ex2((st.x - m) * c);
                    const float4 v = ld_cluster4(cluster_addr(base + part_at(r, lane), k));
                    l += f * st.y;
                    o[0] += f * v.x;
                    o[1] += f * v.y;
                    o[2] += f * v.z;
                    o[3] += f * v.w;
                }
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const long long at = (s.q0 + row) * p.H + h;
                reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o_out) + at * LAT_V)[lane] =
                    make_uint2(pack2<FP16>(o[0] * inv, o[1] * inv), pack2<FP16>(o[2] * inv, o[3] * inv));
                if (lane == 0 && p.lse_out) p.lse_out[at] = l == 0.f ? -INFINITY : m * p.scale + logf(l);
            }
        }
        __syncwarp();
        cluster_barrier();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tmem, 512);
    if (tid == 0 && *failed) set_status(p.status, STATUS_TIMEOUT);
}

template <bool FP16, int SPLIT>
cudaError_t launch(const LatentParams& p, const FwdMaps& maps, int slots, int ranks, cudaStream_t stream) {
    const auto kernel = latent_fwd_kernel<FP16, SPLIT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)F_SMEM);
    if (e != cudaSuccess) return e;
    if (SPLIT == SHARED) {   // (the kernel behind it takes its records as they are)
        latent_share_kernel<<<1, SHARE_SLOTS, 0, stream>>>(p, slots);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute attr[1];
    if (SPLIT == CLUSTER) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)ranks;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
    } else {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((SPLIT == SHARED ? share_items(slots, p.H) : slots * ranks) * p.H));
    cfg.blockDim = dim3(FWD_THREADS);
    cfg.dynamicSmemBytes = F_SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = SPLIT == WHOLE ? 0 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel, p, maps, slots);
    if (e != cudaSuccess || SPLIT != SHARED) return e;
    cfg.gridDim = dim3((unsigned)(share_pairs(p.H) * p.H), LAT_V / 16);
    cfg.blockDim = dim3(FWD_ROWS);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, latent_share_join_kernel<FP16>, p, slots);
}

// Few query tiles on long keys: a cluster for each tile pair, as large as leaves every CTA of every cluster an SM
// (measured with some pairs missing or short, hence the third above 152).  Without / by two / by four, in us:
// 512 queries on 8192 keys, 16 heads (48 pairs) 115 / 72 / 43, 32 heads 118 / 76 / 84; 256 on 2048, 8 heads
// 35 / 31 / 22; one on 4096, 32 heads 49 / 31 / 23.  More pairs, or fewer keys, lose: 2 x 2048 on themselves,
// 8 heads (144 pairs) 37 / 56 / 70; 4 x 1024, 4 heads (80) 22 / 26 / 34.
int cluster_of(long long rows_k, int N, int slots, int H) {
    const long long pairs = (long long)slots * H;
    return rows_k / N < 2048 ? 1 : pairs * 4 <= 200 ? 4 : pairs * 2 <= 200 ? 2 : 1;
}

// Whether tile pairs of packed sequences may be shared by the device's choice: two pairs an SM at most (more fill the
// gaps themselves: 4 x 2048 on themselves, 16 heads, 576 pairs 80 us without and 87 with; 2 x 4096 125 / 130; 512, 129,
// 1, 1000 on 8192, 4039, 3000, 1000 at 32 heads, 320 pairs 137 / 131), and keys for a pair of 64 steps, 120 us, beside
// which the 5 us are little (2 x 2048 on themselves, 8 heads 35 / 41).
bool shares(int Tk, int slots, int H, int N) {
    return N > 1 && Tk >= 64 * LAT_TILE && (long long)slots * H <= 304 && slots <= SHARE_SLOTS && H <= SHARE_PARTS / 2 &&
           cluster_of(Tk, N, slots, H) == 1;
}

}  // namespace

// Bytes behind the status header that let the forward share key ranges: items, entries, parts; 0 where it would not.
unsigned long long latent_share_bytes(int B, int Tq, int Tk, int H, int N) {
    if (B != 1 || !shares(Tk, latent_slots(true, Tq, N, FWD_ROWS), H, N)) return 0;
    return LATENT_SHARE_ITEMS * 16ull + SHARE_PARTS * SHARE_FLOATS * 4ull;
}

cudaError_t launch_latent_fwd(const LatentParams& p, bool fp16, cudaStream_t stream) {
    const bool varlen = p.cu_q != nullptr;
    const long long rows_q = varlen ? p.Tq : (long long)p.N * p.Tq, rows_k = varlen ? p.Tk : (long long)p.N * p.Tk;
    FwdMaps maps;
    // without keys nothing is loaded: any valid tensor does
    const void* kv = rows_k > 0 ? p.kv : p.q;
    const void* pe = rows_k > 0 ? p.k_pe : p.q;
    if (!latent_row_map(&maps.q, p.q, LAT_QK, p.H, rows_q, (long long)p.H * LAT_QK, LAT_TILE) ||
        !latent_row_map(&maps.kv, kv, LAT_KV, p.H, rows_k > 0 ? rows_k : 1, (long long)p.H * LAT_KV, LAT_TILE) ||
        !latent_row_map(&maps.pe, pe, LAT_P, 1, rows_k > 0 ? rows_k : 1, p.k_pe_stride, LAT_TILE))
        return cudaErrorInvalidValue;
    const int slots = latent_slots(varlen, p.Tq, p.N, FWD_ROWS);
    const int ranks = cluster_of(rows_k, p.N, slots, p.H);
    if (ranks > 1)
        return fp16 ? launch<true, CLUSTER>(p, maps, slots, ranks, stream) : launch<false, CLUSTER>(p, maps, slots, ranks, stream);
    if (p.share_items != nullptr)
        return fp16 ? launch<true, SHARED>(p, maps, slots, 1, stream) : launch<false, SHARED>(p, maps, slots, 1, stream);
    return fp16 ? launch<true, WHOLE>(p, maps, slots, 1, stream) : launch<false, WHOLE>(p, maps, slots, 1, stream);
}

}  // namespace kda
