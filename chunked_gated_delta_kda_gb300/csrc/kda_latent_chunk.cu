// Attention of a chunk of new tokens over the paged latent cache
// (kda_latent_chunk), with its C entry point.  See include/kda.h for the
// contract.
//
// Keys and values are expanded from the cached rows, for all heads, into the
// workspace, and the expanded forward runs on them.  A pair of a query and a
// key then costs 640 operations a head beside 2176 in the absorbed form, and
// the expansion 262144 for each key and head, so it is cheaper from some 170
// new tokens a sequence on (where fewer are usual, kda_latent_decode serves).
//
// The expansion is a matrix product whose first operand is gathered page by
// page:  [k_jh | v_jh] = W_h c_j,  512 channels.  A pair of SMs makes 256 rows
// j of one head at a time, 128 rows each; all (pair of tiles, head) items form
// one line, heads inside tiles, cut into equal ranges, one a pair.  The rows
// stay in shared memory for all heads of the range, and of W_h each SM loads
// and reads half.
//
// 65536 rows, 16 heads: 170 us, 1620 TFLOP/s, as fast as the 537 MB that it
// writes (a fill alone takes 135 us) and the power limit allow: without the
// stores 140, without the loads 159.  16231 rows of four sequences on pages of
// 16: 53 us, tensor cores 65 % busy while SMs have work.  On the way there:
// 206 us with a whole W_h in every SM, 193 with pairs, 187 with rows leaving as
// whole lines by way of shared memory (a thread a row before), 170 with a
// tile of a head in one piece ([H, rows, 256]; [rows, H, 256] before).
// The attention behind it takes 447 us, 1440 TFLOP/s of the mask's pairs.
//   warps 0-7  the product's rows out of tensor memory, rounded, to the
//              workspace (two accumulators of 256 columns take turns)
//   warp 8     the first SM's issues the products of both
//   warp 9     loads: a tile's rows (eight slabs of 64 channels), and half of
//              W_h in slabs of 64 channels through a ring
#include <cmath>
#include <cstdint>

#include "kda.h"
#include "kda_latent_mma.cuh"

namespace kda {

uint32_t debug_wait_limit();
cudaError_t launch_latent_fwd(const LatentParams& p, bool fp16, cudaStream_t stream);
unsigned long long latent_share_bytes(int B, int Tq, int Tk, int H, int N);

namespace {

struct ChunkParams {
    const void* cache;          // [num_pages * page_size, 576]
    const int32_t* table;       // [N, width]
    const int32_t* lens;        // [N]
    const int32_t* cu_q;        // [N + 1]
    int32_t* cu_k;              // [N + 1] expanded rows before each sequence
    int32_t* tiles;             // [N + 1] tiles before each sequence
    void* kv;                   // [H, num_keys, 256]: a tile of a head is 64 KiB in one piece
    void* pe;                   // [num_keys, 64]
    void* k_lo;                 // [H, lo_rows, 128]
    int32_t* cu_lo;             // [N + 1] rows of k_lo before each sequence's
    long long lo_rows;
    int lo_tiles;
    uint32_t* status;
    int num_pages, page_size, width, num_keys, T, H, N;
    uint32_t wait_limit;
};

struct ChunkMaps {
    CUtensorMap cache, w;
};

// ---- where each sequence's expanded rows and tiles start: one CTA ----
constexpr int PLAN_THREADS = 1024;

// Sum of `mine` over the threads before this one; the CTA's total in `total`.
__device__ __forceinline__ long long threads_before(long long mine, long long& total, long long* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    long long before = x - mine;
    total = 0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    return before;
}

__global__ void __launch_bounds__(PLAN_THREADS) latent_chunk_plan_kernel(const __grid_constant__ ChunkParams p) {
    __shared__ long long sums[PLAN_THREADS / 32];
    const int tid = threadIdx.x;
    const long long most = (long long)p.width * p.page_size;
    long long rows0 = 0, tiles0 = 0, lo0 = 0, all;
    bool bad = false, bad_cu = false;
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
    if (tid < WS_CLEAR / 4) p.status[tid] = 0u;
    for (int base = 0; base < p.N; base += blockDim.x) {
        const int n = base + tid;
        long long rows = 0, lq = 0;
        if (n < p.N) {
            const int a = p.cu_q[n], b = p.cu_q[n + 1], len = p.lens[n];
            bad_cu |= a < 0 || b < a || b > p.T || (n == 0 && a != 0);
            if (b > a) {
                bad |= len < 0 || len > most;
                rows = max(0ll, min((long long)len, most));
                lq = (long long)b - a;
            }
        }
        const long long before = rows0 + threads_before(rows, all, sums);
        rows0 += all;
        const long long first = min(before, (long long)p.num_keys), last = min(before + rows, (long long)p.num_keys), lk = last - first;
        bad |= lk < rows;
        // tiles; rows of k_lo: those that a sequence's first 256 queries see, or more, where they are few enough
        const long long sees = lk - lq + min(lq, 256ll), limit = (long long)p.lo_tiles * LAT_TILE;
        const long long tiles = (lk + LAT_TILE - 1) / LAT_TILE, lo = sees <= limit ? min(lk, limit) : 0;
        const long long tiles_at = tiles0 + threads_before(tiles, all, sums);
        tiles0 += all;
        const long long lo_at = lo0 + threads_before(lo, all, sums);
        lo0 += all;
        if (n < p.N) {
            p.cu_k[n] = (int)first;
            p.tiles[n] = (int)tiles_at;
            p.cu_lo[n] = (int)lo_at;
        }
    }
    if (tid == 0) {
        p.cu_k[p.N] = (int)min(rows0, (long long)p.num_keys);
        p.tiles[p.N] = (int)tiles0;
        p.cu_lo[p.N] = (int)lo0;
    }
    __syncthreads();                             // the status word is clear
    if (bad) set_status(p.status, STATUS_BAD_PAGE);
    if (bad_cu) set_status(p.status, STATUS_BAD_CU);
}

// ---- the expansion ----
constexpr int EX_THREADS = 320;
constexpr uint32_t EX_SLAB = LAT_TILE * 128;             // 128 rows or columns x 64 channels
constexpr uint32_t SLABS = LAT_C / 64;
constexpr uint32_t EX_RING = 4;
constexpr uint32_t X_A = 0;
constexpr uint32_t X_B = X_A + SLABS * EX_SLAB;
constexpr uint32_t X_STAGE = X_B + EX_RING * EX_SLAB;    // [8 warps] 32 rows x 64 columns
constexpr uint32_t X_AFULL = X_STAGE + 8 * 4096;         // [8] both SMs' slabs have landed (in the first SM)
constexpr uint32_t X_AEMPTY = X_AFULL + 8 * SLABS;       // [8]
constexpr uint32_t X_BFULL = X_AEMPTY + 8 * SLABS;               // [4] (in the first SM)
constexpr uint32_t X_BEMPTY = X_BFULL + 8 * EX_RING;     // [4]
constexpr uint32_t X_DFULL = X_BEMPTY + 8 * EX_RING;     // [2]
constexpr uint32_t X_DEMPTY = X_DFULL + 16;              // [2] (in the first SM)
constexpr uint32_t X_DRAIN = X_DEMPTY + 16;
constexpr uint32_t X_TMEM = X_DRAIN + 8;
constexpr uint32_t X_FAILED = X_TMEM + 4;
constexpr uint32_t X_BYTES = X_FAILED + 4;
constexpr uint32_t X_SMEM = X_BYTES + 1024;
static_assert(X_SMEM <= 232448, "shared memory of one CTA");

// ---- the two SMs of a pair ----
// One product of 256 rows and 256 columns; rows, columns of B and results are half in each SM's memory.
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, Desc a, Desc b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on the barrier at this place in both SMs once the products issued before are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
        "elect.sync r|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(bar)
        : "memory");
}
// A load into this SM's memory that completes on a barrier of either (a cluster address).
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const void* tmap, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A tile of the line: sequence, first row of the tile in it, its rows there.
struct ChunkTile {
    int n, row0, rows, out0;
    int lo0, lo_rows;                            // the tile's first row in k_lo, how many of its rows are there
    __device__ __forceinline__ void find(const ChunkParams& p, int tile, int all) {
        n = row0 = rows = out0 = lo0 = lo_rows = 0;
        if (tile >= all) return;                 // the second of the last pair
        int lo = 0, hi = p.N - 1;                // the last sequence whose tiles start at or before this one
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.tiles[mid] <= tile) lo = mid;
            else hi = mid - 1;
        }
        n = lo;
        row0 = (tile - p.tiles[lo]) * LAT_TILE;
        out0 = p.cu_k[lo] + row0;
        rows = min(LAT_TILE, p.cu_k[lo + 1] - out0);
        lo0 = p.cu_lo[lo] + row0;
        lo_rows = min(rows, p.cu_lo[lo + 1] - lo0);
    }
};

// A warp's 32 rows of 64 16-bit columns (two in a word) to rows `stride` bytes
// apart, the first `rows` of them.  A thread has a row, and rows written from
// there are 32 lines an instruction: they go through 4 KiB of shared memory, a
// row's 16-byte pieces swizzled by the row, and leave as whole 128-byte lines.
__device__ __forceinline__ void store_rows(uint8_t* stage, const uint32_t (&w)[32], uint8_t* out, int stride, int rows, int lane) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) * 16)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = 4 * i + (lane >> 3), c = lane & 7;
        const uint4 x = *reinterpret_cast<const uint4*>(stage + row * 128 + ((c ^ (row & 7)) * 16));
        if (row < rows) *reinterpret_cast<uint4*>(out + row * stride + c * 16) = x;
    }
    __syncwarp();
}

template <bool FP16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(EX_THREADS, 1)
    latent_expand_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ ChunkMaps maps) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;   // at the same place in both SMs
    uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
    volatile uint32_t* failed = reinterpret_cast<volatile uint32_t*>(smem + X_FAILED);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const uint32_t limit = p.wait_limit != 0u ? p.wait_limit : WAIT_LIMIT;
    if (tid == 32) {
        prefetch_map(&maps.cache);
        prefetch_map(&maps.w);
    }
    if (tid == 0) {
        for (uint32_t i = 0; i < SLABS; ++i) {
            mbar_init(base + X_AFULL + 8 * i, 1);
            mbar_init(base + X_AEMPTY + 8 * i, 1);
        }
        for (uint32_t i = 0; i < EX_RING; ++i) {
            mbar_init(base + X_BFULL + 8 * i, 1);
            mbar_init(base + X_BEMPTY + 8 * i, 1);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(base + X_DFULL + 8 * i, 1);
            mbar_init(base + X_DEMPTY + 8 * i, 16);
        }
        mbar_init(base + X_DRAIN, 1);
        *failed = 0u;
        fence_mbar_init();
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base + X_TMEM) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_barrier();                                             // both SMs' barriers and tensor memory are there
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + X_TMEM);
    // The plan; then what follows may begin.  In this order: latent_share_kernel runs beside this kernel, reads the plan's
    // cu_k and writes its records over those that the call before has read, with no wait of its own in front.
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
    const int all_tiles = p.tiles[p.N];
    const long long total = (long long)((all_tiles + 1) / 2) * p.H;
    const long long pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    const long long first = total * pair / pairs, last = total * (pair + 1) / pairs;   // of both SMs alike, maybe none
    const int tile0 = (int)(first / p.H), h0 = (int)(first - (long long)tile0 * p.H);
    const uint32_t lead = cluster_addr(base, 0);                   // the first SM's memory

    if (warp == 9) {
        const int box = min(p.page_size, 64), boxes = LAT_TILE / box;
        const int nowhere = p.num_pages * p.page_size;             // rows from here on read as zeros
        uint32_t loads = 0, tiles = 0;
        int tile = tile0, h = h0;
        bool ok = true, bad = false;
        for (long long i = first; i < last && ok; ++i) {
            const bool fresh = i == first || h == 0;
            int row = nowhere;
            if (fresh) {
                ChunkTile t;
                t.find(p, 2 * tile + (int)rank, all_tiles);
                if (lane < boxes && lane * box < t.rows) {
                    const int key = t.row0 + lane * box, page = p.table[(long long)t.n * p.width + key / p.page_size];
                    if (page >= 0 && page < p.num_pages) row = page * p.page_size + key % p.page_size;
                    else bad = true;
                }
                ++tiles;
            }
            for (uint32_t c = 0; c < SLABS; ++c, ++loads) {
                const uint32_t slot = loads % EX_RING;
                if (fresh) {                                       // a slab of the tile's rows as the last head of the tile before frees it
                    if (tiles > 1 && !wait_warp(base + X_AEMPTY + 8 * c, tiles & 1, limit, failed)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0 && lane == 0) mbar_arrive_expect_tx(base + X_AFULL + 8 * c, 2 * EX_SLAB);
                    __syncwarp();
                    if (lane < boxes)
                        tma_load_pair(base + X_A + c * EX_SLAB + lane * box * 128, &maps.cache, 64 * c, 0, row, lead + X_AFULL + 8 * c);
                }
                if (loads >= EX_RING && !wait_warp(base + X_BEMPTY + 8 * slot, (loads / EX_RING - 1) & 1, limit, failed)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    if (rank == 0) mbar_arrive_expect_tx(base + X_BFULL + 8 * slot, 2 * EX_SLAB);
                    tma_load_pair(base + X_B + slot * EX_SLAB, &maps.w, 64 * c, 0, h * LAT_KV + (int)rank * LAT_TILE,
                                  lead + X_BFULL + 8 * slot);
                }
                __syncwarp();
            }
            if (++h == p.H) h = 0, ++tile;
        }
        if (bad) set_status(p.status, STATUS_BAD_PAGE);
    } else if (warp == 8) {
        if (rank == 0) {
            const uint32_t id = idesc_f16(FP16 ? T_F16 : T_BF16, 256, 256, false, false);
            uint32_t loads = 0, tiles = 0, item = 0;
            int h = h0;
            bool ok = true;
            for (long long i = first; i < last && ok; ++i, ++item) {
                const bool fresh = i == first || h == 0;
                const uint32_t buf = item & 1;
                if (fresh) ++tiles;
                if (item >= 2 && !wait_warp(base + X_DEMPTY + 8 * buf, (item / 2 - 1) & 1, limit, failed)) break;
                tc_fence_after();
                for (uint32_t c = 0; c < SLABS; ++c, ++loads) {
                    const uint32_t slot = loads % EX_RING;
                    if (fresh && !wait_warp(base + X_AFULL + 8 * c, (tiles - 1) & 1, limit, failed)) ok = false;
                    if (ok && !wait_warp(base + X_BFULL + 8 * slot, (loads / EX_RING) & 1, limit, failed)) ok = false;
                    if (!ok) break;
                    const Desc a = desc_k(base + X_A + c * EX_SLAB), b = desc_k(base + X_B + slot * EX_SLAB);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) mma_pair(tmem + 256 * buf, a + 2 * ks, b + 2 * ks, id, c + ks > 0);
                    commit_pair(base + X_BEMPTY + 8 * slot);
                    if (h == p.H - 1) commit_pair(base + X_AEMPTY + 8 * c);
                }
                if (!ok) break;
                commit_pair(base + X_DFULL + 8 * buf);
                if (++h == p.H) h = 0;
            }
            commit_pair(base + X_DRAIN);
        }
        // every product is done, and has been signalled, before the tensor and shared memory go
        mbar_wait(base + X_DRAIN, 0, DRAIN_LIMIT);
    } else {
        const int quarter = warp & 3, half = warp >> 2, r0 = quarter * 32, r = r0 + lane;
        const uint32_t at = tmem + ((uint32_t)quarter << 21);      // this warp's lanes
        uint8_t* stage = smem + X_STAGE + warp * 4096;
        ChunkTile t;
        int tile = tile0, h = h0;
        uint32_t item = 0;
        for (long long i = first; i < last; ++i, ++item) {
            if (i == first || h == 0) t.find(p, 2 * tile + (int)rank, all_tiles);
            if (h == 0 && half == 0 && r < t.rows) {               // the positional channels, once for all heads
                const int key = t.row0 + r, page = p.table[(long long)t.n * p.width + key / p.page_size];
                const bool there = page >= 0 && page < p.num_pages;
                const uint4* from = reinterpret_cast<const uint4*>(
                    static_cast<const uint16_t*>(p.cache) + ((long long)(there ? page : 0) * p.page_size + key % p.page_size) * LAT_ROW + LAT_C);
                uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.pe) + (long long)(t.out0 + r) * LAT_P);
#pragma unroll
                for (int k = 0; k < LAT_P / 8; ++k) to[k] = there ? __ldg(from + k) : make_uint4(0, 0, 0, 0);
            }
            const uint32_t buf = item & 1;
            if (!wait_warp(base + X_DFULL + 8 * buf, (item / 2) & 1, limit, failed)) break;
            tc_fence_after();
            uint8_t* out = static_cast<uint8_t*>(p.kv) + ((long long)h * p.num_keys + t.out0 + r0) * (LAT_KV * 2);
            uint8_t* out_lo = static_cast<uint8_t*>(p.k_lo) + (h * p.lo_rows + t.lo0 + r0) * (LAT_N * 2);
#pragma unroll
            for (int k = 0; k < 2; ++k) {                          // 64 columns of the key, 64 of the value
                const int b = half + 2 * k;
                float x[2][32];
                uint32_t w[32];
                tmem_ld32(at + 256 * buf + 64 * b, x[0]);
                tmem_ld32(at + 256 * buf + 64 * b + 32, x[1]);
                tmem_ld_wait();
                if (k == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_cluster(lead + X_DEMPTY + 8 * buf);
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) w[e] = pack2<FP16>(x[e >> 4][2 * e & 31], x[e >> 4][(2 * e & 31) + 1]);
                store_rows(stage, w, out + 128 * b, LAT_KV * 2, t.rows - r0, lane);
                if (k == 0 && t.lo_rows > r0) {                    // what the keys lose in rounding, nothing where they are infinite
                    auto lost = [](float x, float hi) { return fabsf(hi) < INFINITY ? x - hi : 0.f; };
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float2 hi = unpack2<FP16>(w[e]);
                        w[e] = pack2<FP16>(lost(x[e >> 4][2 * e & 31], hi.x), lost(x[e >> 4][(2 * e & 31) + 1], hi.y));
                    }
                    store_rows(stage, w, out_lo + 128 * b, LAT_N * 2, t.lo_rows - r0, lane);
                }
            }
            if (++h == p.H) h = 0, ++tile;
        }
    }
    tc_fence_before();
    __syncthreads();
    // The products have waited for every copy, unless a role has given up: copies in flight then get 100 us to land.
    if (*failed)
        for (int i = 0; i < 100; ++i) __nanosleep(1000);
    cluster_barrier();                                             // neither SM is used by the other any more
    tc_fence_after();
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    if (tid == 0 && *failed) set_status(p.status, STATUS_TIMEOUT);
}

unsigned long long up256(unsigned long long b) { return (b + 255ull) / 256ull * 256ull; }

// Queries that see at most this many tiles of keys get them as two numbers a
// channel.  A key's rounding (2^-9 of it in bf16) reaches the scores, and their
// log-sum-exp averages it over the keys that count (scores of unit variance: a
// relative error of 8e-5 at 237 keys, 6e-6 at 2100, 3.5e-6 at 8192), so beyond
// that the second numbers are left out: they add 40 % to the products of a pair
// and 20 % to the expansion (8 x 1024 tokens on 4096 rows, H=16: 456 us with
// them, 331 without).  fp16 rounds eight times finer (1e-5 at 129 keys, 6e-6 at
// 300).
int lo_tiles(bool fp16) { return fp16 ? 2 : 16; }

struct ChunkLayout {
    unsigned long long cu, tiles, cu_lo, kv, pe, lo, bytes;
    long long lo_rows;
    ChunkLayout(int T, int num_keys, int H, int N) {
        cu = WS_HEADER + up256(latent_share_bytes(1, T, num_keys, H, N));
        tiles = cu + up256((N + 1ull) * 4ull);
        cu_lo = tiles + up256((N + 1ull) * 4ull);
        kv = cu_lo + up256((N + 1ull) * 4ull);
        pe = kv + (unsigned long long)num_keys * H * LAT_KV * 2ull;
        lo = pe + up256((unsigned long long)num_keys * LAT_P * 2ull);
        const long long most = (long long)N * lo_tiles(false) * LAT_TILE;
        lo_rows = num_keys < most ? num_keys : most;
        bytes = lo + (unsigned long long)lo_rows * H * LAT_N * 2ull;
    }
};

// (the last line: as kda_latent_fwd, a CTA a tile slot and head, in one dimension of a grid)
bool sizes_ok(int T, int num_keys, int H, int N) {
    return T >= 0 && num_keys >= 0 && H >= 1 && N >= 1 && H <= 65535 && N <= 65535 &&
           ((long long)(T > num_keys ? T : num_keys) / LAT_TILE + N) * H < (1ll << 31);
}

bool off(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

}  // namespace

}  // namespace kda

extern "C" {

size_t kda_latent_chunk_workspace_bytes(int T, int num_keys, int H, int N) {
    return kda::sizes_ok(T, num_keys, H, N) ? (size_t)kda::ChunkLayout(T, num_keys, H, N).bytes : 0;
}

kda_status kda_latent_chunk(const void* q, const void* cache, int num_pages, int page_size,
                            const int32_t* block_table, int table_width, const int32_t* seq_lens, const void* w_up,
                            float scale, const int32_t* cu_seqlens_q, int num_keys, void* o, float* lse, int T, int H,
                            int N, unsigned flags, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    using namespace kda;
    if (!sizes_ok(T, num_keys, H, N) || (flags & ~KDA_FLAG_FP16) != 0u) return KDA_ERR_INVALID_ARG;
    if (num_pages < 1 || table_width < 1) return KDA_ERR_INVALID_ARG;
    if (page_size != 16 && page_size != 32 && (page_size < 64 || page_size % 64 != 0)) return KDA_ERR_INVALID_ARG;
    if ((long long)num_pages * page_size >= (1ll << 31) || (long long)table_width * page_size >= (1ll << 31))
        return KDA_ERR_INVALID_ARG;
    if ((T > 0 && (!q || !o)) || !cache || !block_table || !seq_lens || !w_up || !cu_seqlens_q || !workspace)
        return KDA_ERR_INVALID_ARG;
    if (off(q, 16) || off(cache, 16) || off(block_table, 4) || off(seq_lens, 4) || off(w_up, 16) || off(cu_seqlens_q, 4) ||
        off(o, 16) || off(lse, 4) || off(workspace, 256))
        return KDA_ERR_INVALID_ARG;
    const ChunkLayout at(T, num_keys, H, N);
    if (workspace_bytes < at.bytes) return KDA_ERR_INVALID_ARG;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    ChunkParams c{};
    c.cache = cache, c.table = block_table, c.lens = seq_lens, c.cu_q = cu_seqlens_q;
    c.cu_k = reinterpret_cast<int32_t*>(ws + at.cu), c.tiles = reinterpret_cast<int32_t*>(ws + at.tiles);
    c.cu_lo = reinterpret_cast<int32_t*>(ws + at.cu_lo), c.k_lo = ws + at.lo, c.lo_rows = at.lo_rows, c.lo_tiles = lo_tiles((flags & KDA_FLAG_FP16) != 0u);
    c.kv = ws + at.kv, c.pe = ws + at.pe, c.status = reinterpret_cast<uint32_t*>(ws);
    c.num_pages = num_pages, c.page_size = page_size, c.width = table_width, c.num_keys = num_keys;
    c.T = T, c.H = H, c.N = N, c.wait_limit = debug_wait_limit();
    LatentParams p{};
    if (latent_share_bytes(1, T, num_keys, H, N) > 0) {
        p.share_items = reinterpret_cast<int4*>(ws + WS_HEADER);
        p.share_parts = reinterpret_cast<float*>(ws + WS_HEADER + LATENT_SHARE_ITEMS * 16ull);
    }
    p.q = q, p.kv = c.kv, p.k_pe = c.pe, p.k_pe_stride = LAT_P, p.o_out = o, p.lse_out = lse;
    p.cu_q = cu_seqlens_q, p.cu_k = c.cu_k, p.status = c.status;
    p.scale = scale > 0.f && !std::isnan(scale) ? scale : 1.0f / std::sqrt((float)LAT_QK);
    p.k_lo = c.k_lo, p.cu_lo = c.cu_lo, p.lo_rows = at.lo_rows, p.lo_tiles = c.lo_tiles;
    p.Tq = T, p.Tk = num_keys, p.H = H, p.N = N, p.causal = 1, p.chunk = 1, p.wait_limit = debug_wait_limit();

    // each kernel may be set up while the one before it runs, which it waits for
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3((unsigned)(N < PLAN_THREADS ? (N + 31) / 32 * 32 : PLAN_THREADS));
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (!succeeded(cudaLaunchKernelEx(&cfg, latent_chunk_plan_kernel, c))) return KDA_ERR_CUDA;
    if (T == 0) return KDA_OK;
    const bool fp16 = (flags & KDA_FLAG_FP16) != 0u;
    if (num_keys > 0) {
        ChunkMaps maps;
        if (!latent_row_map(&maps.cache, cache, LAT_ROW, 1, (long long)num_pages * page_size, LAT_ROW, page_size < 64 ? page_size : 64) ||
            !latent_row_map(&maps.w, w_up, LAT_C, 1, (long long)H * LAT_KV, LAT_C, LAT_TILE))
            return KDA_ERR_CUDA;
        const auto kernel = fp16 ? latent_expand_kernel<true> : latent_expand_kernel<false>;
        if (!succeeded(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)X_SMEM))) return KDA_ERR_CUDA;
        const long long items = (((long long)num_keys / LAT_TILE + N + 1) / 2) * H;
        cfg.gridDim = dim3(2u * (unsigned)(items < 76 ? items : 76));
        cfg.blockDim = dim3(EX_THREADS);
        cfg.dynamicSmemBytes = X_SMEM;
        if (!succeeded(cudaLaunchKernelEx(&cfg, kernel, c, maps))) return KDA_ERR_CUDA;
    }
    return succeeded(launch_latent_fwd(p, fp16, stream)) ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
