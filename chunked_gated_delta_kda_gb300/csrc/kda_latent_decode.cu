// Absorbed latent attention over the paged cache (kda_latent_decode).
//
// The cached rows serve up to 64 rows (token, head) of a sequence, as keys with
// their 576 channels and as values with the first 512, so each is read once for
// them and used from shared memory by both products; S H rows of a sequence
// walk its cache ceil(S H / 64) times:
//   S = Q R^T            [rows, 64 keys]       M = 64, K = 576
//   O^T += R_v^T P^T     [512 channels, rows]  four M = 128 blocks, K = 64 keys
// O is kept transposed: its channels fill the lanes of tensor memory whatever
// the number of rows, so 64 rows take half of it, and the second product costs
// what the rows need (16, 32 or 64) instead of a padded 128.
//
// Bound by the cache's bytes: 64 rows of the cache are 72 KiB, about 3100
// cycles of an SM's share of the HBM, beside about 1800 of products (both
// limited by what the tensor core reads from shared memory) and 800 of
// softmax, which overlap.  The lengths are on the device, so the work is
// split there: the 64-key tiles of all (sequence, 64-row block) units form
// one line that is cut into equal ranges, one a CTA, wherever the cuts fall.
// A unit inside one range is finished by its CTA; the parts of a cut one go
// to the workspace with their log-sum-exp and are joined by a second kernel,
// which also writes the empty sequences.
// One token of 256 sequences of 4096, H=32: 208 us, 5.8 TB/s (a tile every 3270
// cycles, 6.5 TB/s, and some 15 us of plan, first loads, parts and join); of
// lengths 1 to 8192 222 us, 5.5 TB/s; of one sequence of 65536, 29 us (23 where
// the same 75 MB are read each time and partly stay in the L2).  64 rows (a
// unit's queries then leave room for two tiles) 64 x 8192 rows of cache 123 us,
// 4.9 TB/s; there, four tiles of 32 keys were slower (145).  128 rows of the
// same 224 us, 2.7 TB/s of the cache and 5.4 of its two walks; 16 sequences of
// 8192 with 7 tokens of 128 heads, 14 walks, 321 us, 6.6 TB/s of all of them.
// P is rounded to the cache's type as an operand of the second product (32-bit
// operands run at half the rate and take twice the room): bf16 o is off by
// 0.0021 of its norm, 0.0017 of that its own rounding; the sums, the maximum and
// the parts are in 32 bits.
//   warps 0-3  softmax (row 16 w + l in lanes l and 16 + l of warp w, half of
//              the keys each: an M = 64 product has its rows in 16 lanes of
//              each quarter of tensor memory), rescaling and output of O
//   warps 4, 5  issue the products, 4 the scores and 5 those with the values:
//              the values' part of a tile must not wait for the next tile's
//              loads, which its end makes room for
//   warp 6     loads (asking besides for pages a few tiles ahead to be brought
//              into the L2 cost time: N=256 L=4096 255 us instead of 215)
#include "kda_latent_decode.cuh"
#include "kda_latent_mma.cuh"

namespace kda {

namespace {

constexpr int DEC_THREADS = 224;
constexpr int KEYS = 64;                                 // keys of a tile
constexpr uint32_t KSLAB = KEYS * 128;                   // 64 channels of a tile
constexpr uint32_t HALF = 4 * KSLAB;                     // 256 latent channels of a tile: the unit of the ring
constexpr float RESCALE_LOG2 = 8.f;

// 64-bit quotient of non-negative numbers that mostly fit 32 bits.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Shared-memory layout for R rows of a unit: Q, P, then the two rings.
template <int R>
struct Lay {
    static constexpr uint32_t NH = R == 64 ? 4 : 5, NE = R == 64 ? 2 : 3;   // 2 or 2.5 tiles in flight
    static constexpr uint32_t Q = 0;                     // 9 slabs of R rows
    static constexpr uint32_t P = Q + 9 * R * 128;
    static constexpr uint32_t RH = P + R * 128;          // halves
    static constexpr uint32_t RE = RH + NH * HALF;       // positional slabs
    static constexpr uint32_t HFULL = RE + NE * KSLAB;
    static constexpr uint32_t HEMPTY = HFULL + 8 * NH;
    static constexpr uint32_t EFULL = HEMPTY + 8 * NH;
    static constexpr uint32_t EEMPTY = EFULL + 8 * NE;
    static constexpr uint32_t QFULL = EEMPTY + 8 * NE;
    static constexpr uint32_t SFULL = QFULL + 8;         // [2]
    static constexpr uint32_t WFULL = SFULL + 16;        // [2] P written
    static constexpr uint32_t VDONE = WFULL + 16;        // second product of a tile done
    static constexpr uint32_t OFREE = VDONE + 8;         // O read out
    static constexpr uint32_t DRAIN = OFREE + 8;
    static constexpr uint32_t FACT = DRAIN + 16;         // [64] floats
    static constexpr uint32_t PLAN = FACT + 256;
    static constexpr uint32_t BYTES = PLAN + 256;
    static constexpr uint32_t SMEM = BYTES + 1024;
    static_assert(SMEM <= 232448, "shared memory of one CTA");
};

struct Plan {
    long long scan[DEC_THREADS / 32];
    long long count;            // tiles of this CTA's range
    int n, mt, k0;              // where it starts
    uint32_t tmem, failed, err;
};

struct DecMaps {
    CUtensorMap q, cache;
};

__device__ __forceinline__ int clipped_len(const DecodeParams& p, int n) {
    const long long most = (long long)p.table_width * p.page_size;
    return (int)max(0ll, min((long long)p.lens[n], most));
}

// A role's walk over the segments of its CTA's range.
struct Walk {
    int n, mt, k0, tiles, cnt, len;
    long long left;             // tiles of the range from this segment on
    bool first;
    __device__ __forceinline__ void set(const DecodeParams& p) {
        len = clipped_len(p, n);
        tiles = (len + KEYS - 1) / KEYS;
        cnt = (int)min((long long)(tiles - k0), left);
    }
    __device__ __forceinline__ Walk(const DecodeParams& p, const Plan& pl)
        : n(pl.n), mt(pl.mt), k0(pl.k0), left(pl.count), first(true) {
        if (left > 0) set(p);
    }
    __device__ __forceinline__ void next(const DecodeParams& p, int mts) {
        left -= cnt;
        first = false;
        if (left <= 0) return;
        k0 = 0;
        if (++mt == mts) {
            // the next sequence that has rows (there is one), 32 looked at together: whole warp
            mt = 0;
            uint32_t there = 0;
            for (++n; n < p.N; n += 32) {
                const int at = n + (int)(threadIdx.x & 31);
                there = __ballot_sync(0xffffffffu, at < p.N && clipped_len(p, at) > 0);
                if (there != 0u) break;
            }
            n += __ffs(there) - 1;
        }
        set(p);
    }
};

// The page of the 64-key tile's box b (`rows` keys), or -1 where its keys are
// past the sequence's end or the page does not exist.
__device__ __forceinline__ int box_page(const DecodeParams& p, const Walk& w, int tile, int b, int rows, int& row) {
    const int key = tile * KEYS + b * rows;
    row = 0;
    if (key >= w.len) return -1;
    const int page = p.table[(long long)w.n * p.table_width + key / p.page_size];
    row = key % p.page_size;
    return page >= 0 && page < p.num_pages ? page : -1;
}

// Whether a page of the segment does not exist (whole warp).
__device__ __forceinline__ bool bad_pages(const DecodeParams& p, const Walk& w, int lane) {
    const int a = w.k0 * KEYS / p.page_size, last = min((w.k0 + w.cnt) * KEYS, w.len) - 1;
    bool bad = false;
    for (int i = a + lane; i <= last / p.page_size; i += 32) {
        const int page = p.table[(long long)w.n * p.table_width + i];
        bad |= page < 0 || page >= p.num_pages;
    }
    return __any_sync(0xffffffffu, bad);
}

// Keys of a tile that exist, as bits.
__device__ __forceinline__ unsigned long long tile_keys(const DecodeParams& p, const Walk& w, int tile, int box) {
    unsigned long long m = 0;
    for (int b = 0; b < KEYS / box; ++b) {
        int row;
        const int have = min(box, w.len - tile * KEYS - b * box);
        if (have > 0 && box_page(p, w, tile, b, box, row) >= 0)
            m |= (have == 64 ? ~0ull : (1ull << have) - 1) << (b * box);
    }
    return m;
}

template <int R, bool FP16>
__global__ void __launch_bounds__(DEC_THREADS, 1)
    latent_decode_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ DecMaps maps,
                         const __grid_constant__ DecodeScratch sc) {
    using L = Lay<R>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
    Plan& plan = *reinterpret_cast<Plan*>(smem + L::PLAN);
    static_assert(sizeof(Plan) <= 256, "plan");
    volatile uint32_t* failed = &plan.failed;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
    const uint32_t limit = p.wait_limit != 0u ? p.wait_limit : WAIT_LIMIT;
    const int rows = p.S * p.H, mts = (rows + R - 1) / R;
    const int box = min(p.page_size, KEYS);

    if (tid == 32) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.q) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.cache) : "memory");
    }
    if (tid == 0) {
        for (uint32_t i = 0; i < L::NH; ++i) {
            mbar_init(base + L::HFULL + 8 * i, 1);
            mbar_init(base + L::HEMPTY + 8 * i, 1);
        }
        for (uint32_t i = 0; i < L::NE; ++i) {
            mbar_init(base + L::EFULL + 8 * i, 1);
            mbar_init(base + L::EEMPTY + 8 * i, 1);
        }
        mbar_init(base + L::QFULL, 1);
        mbar_init(base + L::SFULL, 1);
        mbar_init(base + L::SFULL + 8, 1);
        mbar_init(base + L::WFULL, 4);
        mbar_init(base + L::WFULL + 8, 4);
        mbar_init(base + L::VDONE, 1);
        mbar_init(base + L::OFREE, 4);
        mbar_init(base + L::DRAIN, 1);
        mbar_init(base + L::DRAIN + 8, 1);
        plan.failed = 0u;
        plan.err = 0u;
        plan.count = 0;
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 4) {
        tmem_alloc(base + L::PLAN + (uint32_t)offsetof(Plan, tmem), 512);
        tmem_relinquish();
    }
    // ---- the line of tiles, and this CTA's part of it ----
    {
        const int per = (p.N + DEC_THREADS - 1) / DEC_THREADS;
        const int a = min(p.N, tid * per), b = min(p.N, a + per);
        long long sum = 0;
        bool bad = false;
        for (int n = a; n < b; ++n) {
            const int len = clipped_len(p, n);
            bad |= len != p.lens[n];
            sum += (long long)((len + KEYS - 1) / KEYS) * mts;
        }
        long long x = sum;
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) plan.scan[warp] = x;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        long long before = 0, total = 0;
        for (int w = 0; w < DEC_THREADS / 32; ++w) {
            if (w < warp) before += plan.scan[w];
            total += plan.scan[w];
        }
        const long long g = min((long long)gridDim.x, total);
        long long at = before + x - sum;               // tiles before sequence a
        if (cta == 0) {
            if (bad) atomicOr(&plan.err, STATUS_BAD_PAGE);
            long long pos = at;
            for (int n = a; n < b; ++n) {
                sc.prefix[n] = pos;
                pos += (long long)((clipped_len(p, n) + KEYS - 1) / KEYS) * mts;
            }
            if (tid == 0) sc.prefix[p.N] = total;
        }
        if (cta < g) {
            const long long lo = quotient(cta * total, g), hi = quotient((cta + 1) * total, g);
            if (lo >= at && lo < at + sum) {           // one thread: the range starts in its sequences
                int n = a;
                for (;; ++n) {
                    const int t = (clipped_len(p, n) + KEYS - 1) / KEYS;
                    if (lo < at + (long long)t * mts) {
                        plan.n = n;
                        plan.mt = (int)quotient(lo - at, t);
                        plan.k0 = (int)(lo - at - (long long)plan.mt * t);
                        break;
                    }
                    at += (long long)t * mts;
                }
                plan.count = hi - lo;
            }
        }
        __syncthreads();
    }
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&plan.tmem);
    const uint32_t t_s = tmem + 256;                   // S: two buffers of 64 columns; O: columns [0, 4 R)

    if (warp == 6) {
        // ---- loads ----
        uint32_t ih = 0, ie = 0;                       // halves and positional slabs asked for
        bool ok = true;
        const int nbox = KEYS / box;
        const int b = lane % nbox, c = lane / nbox;    // this lane's box and slab (nbox <= 4: of 8 or more)
        for (Walk w(p, plan); w.left > 0 && ok; w.next(p, mts)) {
            bool bad = false;
            int row, page = box_page(p, w, w.k0, b, box, row);
            for (int k = 0; k < w.cnt && ok; ++k) {
                const int tile = w.k0 + k;
                const bool have = page >= 0;
                bad |= !have && tile * KEYS + b * box < w.len;
                const int at = page * p.page_size + row;
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, have && c == 0)) * (uint32_t)box * 128u;
                if (k + 1 < w.cnt) page = box_page(p, w, tile + 1, b, box, row);
#pragma unroll
                for (int part = 0; part < 3 && ok; ++part) {   // two halves, then the positional slab
                    const uint32_t i = part < 2 ? ih : ie, depth = part < 2 ? L::NH : L::NE;
                    const uint32_t full = base + (part < 2 ? L::HFULL : L::EFULL) + 8 * (i % depth);
                    if (i >= depth)
                        ok = wait_warp(base + (part < 2 ? L::HEMPTY : L::EEMPTY) + 8 * (i % depth), (i / depth - 1) & 1, limit,
                                       failed);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(full, bytes * (part < 2 ? 4u : 1u));
                    __syncwarp();
                    const uint32_t dst = base + (part < 2 ? L::RH + (i % depth) * HALF : L::RE + (i % depth) * KSLAB) +
                                         (uint32_t)c * KSLAB + (uint32_t)(b * box) * 128u;
                    if (have && c < (part < 2 ? 4 : 1)) tma_load_3d(dst, &maps.cache, 256 * part + 64 * c, 0, at, full);
                    if (part < 2) ++ih;
                    else ++ie;
                }
            }
            if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&plan.err, STATUS_BAD_PAGE);
        }
        // every copy issued here has landed before the CTA ends
        for (uint32_t k = ih > L::NH ? ih - L::NH : 0; k < ih; ++k)
            mbar_wait(base + L::HFULL + 8 * (k % L::NH), (k / L::NH) & 1, DRAIN_LIMIT);
        for (uint32_t k = ie > L::NE ? ie - L::NE : 0; k < ie; ++k)
            mbar_wait(base + L::EFULL + 8 * (k % L::NE), (k / L::NE) & 1, DRAIN_LIMIT);
    } else if (warp >= 4) {
        // ---- products ----
        const MmaType ty = FP16 ? T_F16 : T_BF16;
        const uint32_t id_s = idesc_f16(ty, 64, KEYS, false, false), id_o = idesc_f16(ty, 128, R, true, false);
        uint32_t g = 0, seg = 0;                       // tiles and segments so far
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = ok && wait_warp(base + bar, parity, limit, failed);
            return ok;
        };
        auto half = [&](uint32_t i) { return base + L::RH + (i % L::NH) * HALF; };
        if (warp == 4) {
            for (Walk w(p, plan); w.left > 0 && ok; w.next(p, mts), ++seg) {
                // A lowered limit runs out here one poll early, and a limit of one at once: what it is lowered for is seen
                // however long the hardware suspends a poll.  (Everywhere, a loop that may not run at all costs 1% here,
                // 3% in the forward.)
                ok = wait_warp(base + L::QFULL, seg & 1, p.wait_limit != 0u ? limit - 1u : limit, failed);
                if (!ok) break;
                for (int k = 0; k < w.cnt && ok; ++k, ++g) {
                    // S's buffer is free once the weights of the tile before the last are written
                    if (g >= 2 && !wait(L::WFULL + 8 * (g & 1), ((g - 2) >> 1) & 1)) break;
                    tc_fence_after();
#pragma unroll
                    for (int part = 0; part < 3; ++part) {
                        const uint32_t i = part < 2 ? 2 * g + part : g, depth = part < 2 ? L::NH : L::NE;
                        if (!wait((part < 2 ? L::HFULL : L::EFULL) + 8 * (i % depth), (i / depth) & 1)) break;
                        const Desc a = desc_k(base + L::Q + 4 * part * R * 128);
                        const Desc b = desc_k(part < 2 ? half(i) : base + L::RE + (i % depth) * KSLAB);
#pragma unroll
                        for (int ks = 0; ks < (part < 2 ? 16 : 4); ++ks)
                            mma_ss(t_s + 64 * (g & 1), a + ((ks >> 2) * (R * 8) + (ks & 3) * 2),
                                   b + ((ks >> 2) * (KSLAB / 16) + (ks & 3) * 2), id_s, part + ks > 0);
                    }
                    if (!ok) break;
                    mma_commit_warp(base + L::SFULL + 8 * (g & 1));
                    mma_commit_warp(base + L::EEMPTY + 8 * (g % L::NE));
                }
            }
        } else {
            for (Walk w(p, plan); w.left > 0 && ok; w.next(p, mts), ++seg) {
                const bool gaps = bad_pages(p, w, lane);
                for (int k = 0; k < w.cnt; ++k, ++g) {
                    if (!wait(L::WFULL + 8 * (g & 1), (g >> 1) & 1)) break;
                    if (k == 0 && seg > 0 && !wait(L::OFREE, (seg - 1) & 1)) break;
                    tc_fence_after();
                    const int tile = w.k0 + k;
                    if (gaps || (tile + 1) * KEYS > w.len) {
                        // rows that do not exist hold whatever was there: zero weights must meet zeros
                        uint8_t* at = smem + (half(2 * g) - base) + (lane >> 3) * KSLAB + (lane & 7) * 16;
                        const int other = (int)(half(2 * g + 1) - half(2 * g));
                        // (one sequence of 200, H=16: 10.6 us; 15.4 with a test of each of the 64 rows)
                        auto clear = [&](int r) {
                            *reinterpret_cast<uint4*>(at + r * 128) = make_uint4(0, 0, 0, 0);
                            *reinterpret_cast<uint4*>(at + r * 128 + other) = make_uint4(0, 0, 0, 0);
                        };
                        if (gaps) {
                            for (unsigned long long none = ~tile_keys(p, w, tile, box); none != 0ull; none &= none - 1)
                                clear(__ffsll(none) - 1);
                        } else {
#pragma unroll 8
                            for (int r = w.len - tile * KEYS; r < KEYS; ++r) clear(r);
                        }
                        fence_async_smem();
                        __syncwarp();
                    }
                    const Desc b = desc_k(base + L::P);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {      // O^T: channels 128 c ..
                        const Desc a = desc_mn(half(2 * g + (c >> 1)) + (c & 1) * 2 * KSLAB, KEYS);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) mma_ss(tmem + c * R, a + 128 * ks, b + 2 * ks, id_o, k + ks > 0);
                        if (c & 1) mma_commit_warp(base + L::HEMPTY + 8 * ((2 * g + (c >> 1)) % L::NH));
                    }
                    mma_commit_warp(base + L::VDONE);
                }
            }
        }
        // every product issued here is done before the tensor memory is freed
        mma_commit_warp(base + L::DRAIN + 8 * (warp & 1));
        mbar_wait(base + L::DRAIN + 8 * (warp & 1), 0, DRAIN_LIMIT);
    } else {
        // ---- softmax and output ----
        const float c = p.scale * 1.4426950408889634f;
        const uint32_t quad = (uint32_t)warp << 21;    // this warp's lanes
        const int r = 16 * warp + (lane & 15);         // its row; lanes l and 16 + l have a half of the keys each
        float* fact = reinterpret_cast<float*>(smem + L::FACT);
        uint32_t g = 0, asked = 0;
        bool ok = true;
        // warp 3 asks for the queries: of the next segment as soon as the scores of this one are complete (the loading
        // warp would have to wait for that and could not run ahead into the next segment's rows)
        auto ask = [&](const Walk& w) {
            if (lane == 0) mbar_arrive_expect_tx(base + L::QFULL, 9 * R * 128);
            __syncwarp();
            if (lane < 9)
                tma_load_3d(base + L::Q + lane * R * 128, &maps.q, 64 * lane, 0, w.n * rows + w.mt * R, base + L::QFULL);
            ++asked;
        };
        if (warp == 3 && plan.count > 0) ask(Walk(p, plan));
        for (Walk w(p, plan); w.left > 0 && ok; w.next(p, mts)) {
            const bool gaps = bad_pages(p, w, lane);
            const int gr = w.mt * R + r;
            const int lim = w.len - p.S + 1 + min(gr, rows - 1) / p.H;   // keys [0, lim) are seen
            float m = -INFINITY, l = 0.f;
            for (int k = 0; k < w.cnt && ok; ++k, ++g) {
                ok = wait_warp(base + L::SFULL + 8 * (g & 1), g >> 1 & 1, limit, failed);   // joined with the others' below
                tc_fence_after();
                if (warp == 3 && ok && k + 1 == w.cnt && w.left > w.cnt) {
                    Walk next = w;
                    next.next(p, mts);
                    ask(next);
                }
                const int tile = w.k0 + k;
                float x[32];
                tmem_ld_half32(t_s + 64 * (g & 1) + quad, x);
                tmem_ld_wait();
                const int have = lim - tile * KEYS;
                if (gaps || __any_sync(0xffffffffu, have < KEYS)) {
                    unsigned long long keys = gaps ? tile_keys(p, w, tile, box) : ~0ull;
                    keys &= have >= KEYS ? ~0ull : have > 0 ? (1ull << have) - 1 : 0ull;
                    const uint32_t mine = (uint32_t)(keys >> (lane & 16) * 2);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!(mine >> e & 1)) x[e] = -INFINITY;
                }
                float top = max32(x);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                const bool grown = r < R && (top * c > m * c + RESCALE_LOG2 || (m == -INFINITY && top > m));
                // P's buffer is free, and O stands still, once the tile before is done
                if (k > 0 && ok) ok = wait_warp(base + L::VDONE, (g - 1) & 1, limit, failed);
                if (!bar_and_named(1, 128, ok && !grown)) {
                    ok = bar_and_named(1, 128, ok);
                    if (!ok) break;
                    tc_fence_after();
                    const float mn = grown ? top : m;
                    const float f = grown ? ex2((m - mn) * c) : 1.f;
                    l *= f;
                    m = mn;
                    if (k > 0) {
                        if (lane < 16) fact[r] = f;
                        bar_and_named(1, 128, true);
#pragma unroll 1
                        for (int b = 0; b < 4 * R; b += 16) {
                            float o[16];
                            tmem_ld16(tmem + quad + b, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= fact[(b + e) % R];
#pragma unroll
                            for (int e = 0; e < 16; e += 4)
                                tmem_st4(tmem + quad + b + e, __float_as_uint(o[e]), __float_as_uint(o[e + 1]),
                                         __float_as_uint(o[e + 2]), __float_as_uint(o[e + 3]));
                        }
                        tmem_st_wait();
                    }
                }
                if (r < R) {
                    const float mc = m == -INFINITY ? 0.f : m * c;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float u = x[8 * q + 2 * e], v = x[8 * q + 2 * e + 1];
                            fma2(u, v, c, -mc);
                            u = ex2(u);
                            v = ex2(v);
                            add2(sum[2 * (e & 1)], sum[2 * (e & 1) + 1], u, v);
                            o[e] = pack2<FP16>(u, v);
                        }
                        *reinterpret_cast<uint4*>(smem + L::P + r * 128 + (((q + (lane >> 4) * 4) ^ (r & 7)) * 16)) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(base + L::WFULL + 8 * (g & 1));
            }
            if (ok) ok = wait_warp(base + L::VDONE, (g - 1) & 1, limit, failed);
            ok = bar_and_named(1, 128, ok);
            if (!ok) break;
            tc_fence_after();
            // ---- the segment's rows ----
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const bool whole = w.cnt == w.tiles;
            const int slot = 2 * cta + (w.first ? 0 : 1);
            if (r < R && lane < 16) {
                fact[r] = l == 0.f ? 0.f : 1.f / l;
                const float lse = l == 0.f ? -INFINITY : m * p.scale + logf(l);
                if (whole) {
                    if (gr < rows && p.lse) p.lse[(long long)w.n * rows + gr] = lse;
                } else {
                    sc.lse[slot * R + r] = lse;
                }
            }
            bar_and_named(1, 128, true);
            const int have = min(R, rows - w.mt * R);
            constexpr int RC = R < 32 ? R : 32;        // rows at a time
#pragma unroll 1
            for (int r0 = 0; r0 < R; r0 += RC) {
                float f[RC];
#pragma unroll
                for (int e = 0; e < RC; ++e) f[e] = fact[r0 + e];
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    float o[32];
                    if constexpr (R < 32) tmem_ld16(tmem + quad + b * R, reinterpret_cast<float(&)[16]>(o));
                    else tmem_ld32(tmem + quad + b * R + r0, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < RC; ++e) o[e] = f[e] == 0.f ? 0.f : o[e] * f[e];
                    const int ch = 128 * b + 32 * warp + lane, count = have - r0;
                    if (whole) {
                        uint16_t* out = static_cast<uint16_t*>(p.o) + ((long long)w.n * rows + w.mt * R + r0) * LAT_C + ch;
#pragma unroll
                        for (int e = 0; e < RC; ++e)
                            if (e < count) out[e * LAT_C] = (uint16_t)pack2<FP16>(o[e], 0.f);
                    } else {
                        float* out = sc.o + ((long long)slot * R + r0) * LAT_C + ch;
#pragma unroll
                        for (int e = 0; e < RC; ++e)
                            if (e < count) out[e * LAT_C] = o[e];
                    }
                }
            }
            tc_fence_before();
            bar_and_named(1, 128, true);               // fact is reused by the next segment
            if (lane == 0) mbar_arrive(base + L::OFREE);
        }
        if (asked > 0) mbar_wait(base + L::QFULL, (asked - 1) & 1, DRAIN_LIMIT);   // landed before the CTA ends
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 4) tmem_dealloc(tmem, 512);
    if (tid == 0) sc.err[cta] = plan.err | (plan.failed ? STATUS_TIMEOUT : 0u);
}

// Joins the parts of the units that were cut: lse = log sum exp(lse_i),
// o = sum exp(lse_i - lse) o_i, in a fixed order; writes zeros for empty
// sequences.  WARPS warps share the parts of V groups of 128 channels of a row,
// 8 / WARPS rows a CTA: few units have many parts each, many have few.
template <int WARPS, int V, bool FP16>
__global__ void __launch_bounds__(256) latent_join_kernel(const __grid_constant__ DecodeParams p,
                                                          const __grid_constant__ DecodeScratch sc, int R, int mts, int ctas) {
    constexpr int ROWS = 8 / WARPS;                    // of a CTA
    __shared__ float4 acc[WARPS == 1 ? 1 : 8][32];
    __shared__ float stat[8];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows = p.S * p.H;
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && warp == 0) {
        uint32_t err = 0;
        for (int c = lane; c < ctas; c += 32) err |= sc.err[c];
        err = __reduce_or_sync(0xffffffffu, err);
        if (lane == 0) *p.status = err;
    }
    const int n = blockIdx.x / mts, mt = blockIdx.x % mts;
    const long long total = sc.prefix[p.N], tiles = (sc.prefix[n + 1] - sc.prefix[n]) / mts;
    const long long w0 = sc.prefix[n] + mt * tiles, g = min((long long)ctas, total);
    int c0 = 0, c1 = -1;
    if (tiles > 0) {
        c0 = (int)quotient((w0 + 1) * g - 1, total);
        c1 = (int)quotient((w0 + tiles) * g - 1, total);
        if (c0 == c1) return;
    }
    const int r = blockIdx.y * ROWS + warp / WARPS, part = warp % WARPS;   // r < R
    const bool there = mt * R + r < rows;
    if (WARPS == 1 && !there) return;                  // (warps that work together stay; such rows' parts are not used)
    // the first part of c0's unit is its last segment, unless the unit starts the range
    const int slot0 = 2 * c0 + (tiles > 0 && quotient(c0 * total, g) != w0 ? 1 : 0);
    auto slot_of = [&](int c) { return c == c0 ? slot0 : 2 * c; };
    float m = -INFINITY, l = 0.f;
    float4 o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4* src = reinterpret_cast<const float4*>(sc.o + (long long)r * LAT_C) + blockIdx.z * (32 * V) + lane;
    auto part_of = [&](int c) { return src + (long long)slot_of(c) * R * (LAT_C / 4); };
    // the parts' values do not depend on the weights: ask for them first
    constexpr int BATCH = V == 4 ? 2 : WARPS == 8 ? 20 : 10;   // at once (152 parts of a unit: 20 beside 10 1.3 us less)
    float4 v[BATCH][V];
    auto fetch = [&](int first) {
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            if (first + k * WARPS <= c1) {
#pragma unroll
                for (int e = 0; e < V; ++e) v[k][e] = part_of(first + k * WARPS)[32 * e];
            }
    };
    fetch(c0 + part);
    for (int c = c0 + lane; c <= c1; c += 32) m = fmaxf(m, sc.lse[slot_of(c) * R + r]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    for (int c = c0 + part; c <= c1; c += BATCH * WARPS) {
        if (c > c0 + part) fetch(c);
        const int mine = c + lane * WARPS;             // lane k: the weight of the batch's part k
        float w = 0.f;
        if (lane < BATCH && mine <= c1) {
            const float lse = sc.lse[slot_of(mine) * R + r];
            w = lse == -INFINITY ? 0.f : expf(lse - m);
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            if (c + k * WARPS > c1) break;
            const float wk = __shfl_sync(0xffffffffu, w, k);
            l += wk;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                o[e].x += wk * v[k][e].x;
                o[e].y += wk * v[k][e].y;
                o[e].z += wk * v[k][e].z;
                o[e].w += wk * v[k][e].w;
            }
        }
    }
    if constexpr (WARPS > 1) {
        acc[warp][lane] = o[0];
        if (lane == 0) stat[warp] = l;
        __syncthreads();
        if (part != 0 || !there) return;
        l = 0.f;
        o[0] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < WARPS; ++k) {
            const float4 v = acc[warp + k][lane];
            l += stat[warp + k];
            o[0].x += v.x;
            o[0].y += v.y;
            o[0].z += v.z;
            o[0].w += v.w;
        }
    }
    const long long at = (long long)n * rows + mt * R + r;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint2* out = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + at * LAT_C) + blockIdx.z * (32 * V) + lane;
#pragma unroll
    for (int e = 0; e < V; ++e)
        out[32 * e] = make_uint2(pack2<FP16>(o[e].x * inv, o[e].y * inv), pack2<FP16>(o[e].z * inv, o[e].w * inv));
    if (lane == 0 && blockIdx.z == 0 && p.lse) p.lse[at] = l == 0.f ? -INFINITY : m + logf(l);
}

int unit_rows(int S, int H) { return (long long)S * H <= 16 ? 16 : (long long)S * H <= 32 ? 32 : 64; }

unsigned long long up256(unsigned long long b) { return (b + 255ull) / 256ull * 256ull; }

template <int R, bool FP16>
cudaError_t launch(const DecodeParams& p, const DecMaps& maps, const DecodeScratch& sc, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(latent_decode_kernel<R, FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)Lay<R>::SMEM);
    if (e != cudaSuccess) return e;
    latent_decode_kernel<R, FP16><<<DEC_CTAS, DEC_THREADS, Lay<R>::SMEM, stream>>>(p, maps, sc);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int mts = (p.S * p.H + R - 1) / R;
    // The join may be set up while the last CTAs of the kernel before it run: it waits for them itself.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // By the rows of all units (us a call; 8, 4, 2, 1 warps for 128 channels of a row, 1 for 512).  R = 16, sequences of
    // 2048: 4 of them 12.5 / 12.4 / 13.1 / 14.5 / 19.7, 8 15.0 / 13.5 / 13.4 / 14.1 / 17.5, 24 25.5 / 21.8 / 19.9 / 20.0 /
    // 20.8, 48 45 / 38 / 34.7 / 32.7 / 33.0; R = 64: 1 14.4 / 14.8 / 16.0 / 16.4 / 21.3, 3 17.4 / 15.6 / 17.2 / 17.2 /
    // 22.5, 6 22.6 / 18.8 / 17.5 / 19.4 / 21.7, 12 34.7 / 27.9 / 24.1 / 22.9 / 23.8, 48 96 / 68 / 54 / 47 / 42.
    const int units = p.N * mts;
    const long long of_all = (long long)units * R;
    auto join = [&](auto kernel, int warps, int groups) {
        cfg.gridDim = dim3(units, R / (8 / warps), 4 / groups);
        return cudaLaunchKernelEx(&cfg, kernel, p, sc, R, mts, DEC_CTAS);
    };
    if (of_all <= 64) return join(latent_join_kernel<8, 1, FP16>, 8, 1);
    if (of_all <= 192) return join(latent_join_kernel<4, 1, FP16>, 4, 1);
    if (of_all <= 384) return join(latent_join_kernel<2, 1, FP16>, 2, 1);
    return of_all < 1024 ? join(latent_join_kernel<1, 1, FP16>, 1, 1) : join(latent_join_kernel<1, 4, FP16>, 1, 4);
}

}  // namespace

// Workspace: header, error words of the CTAs, tiles before each sequence, two
// parts a CTA (log-sum-exp and output of each row).
unsigned long long latent_decode_scratch(int N, int S, int H) {
    const unsigned long long r = (unsigned long long)unit_rows(S, H);
    return WS_HEADER + up256(DEC_CTAS * 4ull) + up256((N + 1ull) * 8ull) + up256(2ull * DEC_CTAS * r * 4ull) +
           2ull * DEC_CTAS * r * LAT_C * 4ull;
}

cudaError_t launch_latent_decode(const DecodeParams& p, bool fp16, cudaStream_t stream) {
    const int r = unit_rows(p.S, p.H);
    DecodeScratch sc;
    uint8_t* ws = p.workspace + WS_HEADER;
    sc.err = reinterpret_cast<uint32_t*>(ws);
    ws += up256(DEC_CTAS * 4ull);
    sc.prefix = reinterpret_cast<long long*>(ws);
    ws += up256((p.N + 1ull) * 8ull);
    sc.lse = reinterpret_cast<float*>(ws);
    ws += up256(2ull * DEC_CTAS * r * 4ull);
    sc.o = reinterpret_cast<float*>(ws);
    DecMaps maps;
    const int box = p.page_size < KEYS ? p.page_size : KEYS;
    if (!latent_row_map(&maps.q, p.q, LAT_ROW, 1, (long long)p.N * p.S * p.H, LAT_ROW, r) ||
        !latent_row_map(&maps.cache, p.cache, LAT_ROW, 1, (long long)p.num_pages * p.page_size, LAT_ROW, box))
        return cudaErrorInvalidValue;
    if (r == 16) return fp16 ? launch<16, true>(p, maps, sc, stream) : launch<16, false>(p, maps, sc, stream);
    if (r == 32) return fp16 ? launch<32, true>(p, maps, sc, stream) : launch<32, false>(p, maps, sc, stream);
    return fp16 ? launch<64, true>(p, maps, sc, stream) : launch<64, false>(p, maps, sc, stream);
}

}  // namespace kda
