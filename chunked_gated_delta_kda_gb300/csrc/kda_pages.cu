// Pages that several requests own: forking, freeing, compacting and copying
// (kda_page_fork, kda_page_free, kda_page_compact, kda_page_copy), with their
// C entry points.  See include/kda.h for the contract.
//
// The first three are bookkeeping of a few thousand words whose steps depend
// on each other (owners counted before pages are given back, pages numbered
// before tables are rewritten), so latency bounds them.  Each runs as one
// cluster of eight CTAs with cluster barriers between the steps: one launch
// and no scratch memory, the outputs hold what the steps pass on.  What one
// CTA writes and another reads goes through the L2 (atomics, __stcg, __ldcg).
#include <cstdint>

#include "kda.h"
#include "kda_latent_mma.cuh"

namespace kda {

namespace {

constexpr int PG_CTAS = 8;
constexpr int PG_THREADS = 1024;
constexpr int PG_WARPS = PG_THREADS / 32;
constexpr int PG_ALL = PG_CTAS * PG_THREADS;
constexpr int PG_PER = 8;                        // pages of a thread, in a row
constexpr int PG_CHUNK = PG_THREADS * PG_PER;
constexpr int PG_KEEP = 4;                       // chunks whose masks stay in registers

struct PageParams {
    const int32_t* table;
    int32_t* table_io;
    const int32_t* lens;
    const int32_t* keep;
    const int32_t* parents;
    const int32_t* children;
    const int32_t* refs;
    const int32_t* free_pages;
    int32_t* free_io;
    const int32_t* free_head;
    int32_t* lens_out;
    int32_t* refs_out;
    int32_t* head_out;
    int32_t* free_out;
    int32_t* pairs;
    int32_t* count;
    int32_t* moved;
    uint32_t* status;
    int width, num_pages, num_free, page_size, N, F;
};

// A row's pages, its length clipped to the table's columns.
__device__ __forceinline__ int row_pages(const PageParams& p, int len, bool& bad) {
    const long long most = (long long)p.width * p.page_size;
    bad |= len < 0 || len > most;
    return (int)((max(0ll, min((long long)len, most)) + p.page_size - 1) / p.page_size);
}

template <typename FUNC>
__device__ __forceinline__ void copy_words(const int32_t* from, int32_t* to, int count, int me, FUNC f) {
    if (((reinterpret_cast<uintptr_t>(from) | reinterpret_cast<uintptr_t>(to)) & 15u) == 0) {
        const int quads = count >> 2;
#pragma unroll 4
        for (int i = me; i < quads; i += PG_ALL) {
            const int4 x = __ldg(reinterpret_cast<const int4*>(from) + i);
            __stcg(reinterpret_cast<int4*>(to) + i, make_int4(f(x.x), f(x.y), f(x.z), f(x.w)));
        }
        if (me < (count & 3)) __stcg(to + 4 * quads + me, f(__ldg(from + 4 * quads + me)));
        return;
    }
#pragma unroll 4
    for (int i = me; i < count; i += PG_ALL) __stcg(to + i, f(__ldg(from + i)));
}

__device__ __forceinline__ void fill_words(int32_t* to, int value, int count, int me) {   // on 16 bytes
    for (int i = me; i < count >> 2; i += PG_ALL) __stcg(reinterpret_cast<int4*>(to) + i, make_int4(value, value, value, value));
    if (me < (count & 3)) __stcg(to + (count & ~3) + me, value);
}

// Sum of `mine` over the threads before this one; the CTA's total in `total`.
__device__ __forceinline__ int block_before(int mine, int& total, int* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();                             // the round before is done with the sums
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    const int s = sums[lane];
    total = __reduce_add_sync(0xffffffffu, s);
    return x - mine + __reduce_add_sync(0xffffffffu, lane < warp ? s : 0);
}
static_assert(PG_WARPS == 32, "a lane a warp's sum");

// `mine` of every CTA of the cluster: the sum of those of lower rank, and of
// all.  Has a cluster barrier; `slots` serves one call.
__device__ __forceinline__ int cluster_before(int mine, int& total, int* slots) {
    const uint32_t rank = cluster_rank();
    if (threadIdx.x < PG_CTAS) {
        const uint32_t at = cluster_addr(smem_u32(slots + rank), threadIdx.x);
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(mine) : "memory");
    }
    cluster_barrier();
    int before = 0;
    total = 0;
    for (uint32_t r = 0; r < PG_CTAS; ++r) {
        const int s = slots[r];
        if (r < rank) before += s;
        total += s;
    }
    return before;
}

// ---- fork: a warp an entry ----
// While entries claim their children, lens_out holds i - F at a child of
// length 0 that entry i is the first to have.
__global__ void __cluster_dims__(PG_CTAS, 1, 1) __launch_bounds__(PG_THREADS, 1) page_fork_kernel(const __grid_constant__ PageParams p) {
    __shared__ int sums[PG_WARPS];
    __shared__ int4 entries[PG_THREADS];         // parent (-1: skipped), child, tokens, place among the own pages (-1: none)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)cluster_rank(), me = rank * PG_THREADS + tid;
    const int head = p.free_head[0];
    bool bad = false;
    if (me == 0 && p.status) __stcg(p.status, 0u);
    auto same = [](int x) { return x; };
    copy_words(p.refs, p.refs_out, p.num_pages, me, same);
    copy_words(p.lens, p.lens_out, p.N, me, same);
    cluster_barrier();
    for (int i = me; i < p.F; i += PG_ALL) {
        const int a = p.parents[i], c = p.children[i];
        if (c >= 0 && c < p.N && a >= 0 && a < p.N && p.lens[c] == 0) atomicMin(p.lens_out + c, i - p.F);
    }
    cluster_barrier();
    int taken = 0;
    for (int base = 0; base < p.F; base += PG_THREADS) {
        const int i = base + tid;
        int4 e = make_int4(-1, -1, 0, -1);
        if (i < p.F) {
            const int a = p.parents[i], c = p.children[i];
            if (c >= 0) {
                if (c < p.N && a >= 0 && a < p.N && p.lens[c] == 0 && __ldcg(p.lens_out + c) == i - p.F) {
                    const long long most = (long long)p.width * p.page_size;
                    const int len = p.lens[a];
                    bad |= len < 0 || len > most;
                    e = make_int4(a, c, (int)max(0ll, min((long long)len, most)), -1);
                } else {
                    bad = true;
                }
            }
        }
        const bool part = e.z % p.page_size != 0;
        int total;
        const int before = block_before(part ? 1 : 0, total, sums);
        if (part) e.w = taken + before;
        entries[tid] = e;
        cluster_barrier();                       // every CTA has looked its entries up before lens_out changes
        for (int k = rank * PG_WARPS + warp; k < min(PG_THREADS, p.F - base); k += PG_ALL / 32) {
            const int4 f = entries[k];
            int2 pair = make_int2(-1, -1);
            if (f.x >= 0) {
                const int32_t* from = p.table_io + (long long)f.x * p.width;
                int32_t* to = p.table_io + (long long)f.y * p.width;
                const int full = f.z / p.page_size;
#pragma unroll 4
                for (int col = lane; col < full; col += 32) {
                    int page = from[col];
                    if (page < 0 || page >= p.num_pages) page = -1, bad = true;
                    else atomicAdd(p.refs_out + page, 1);
                    to[col] = page;
                }
                if (f.w >= 0) {
                    const long long at = (long long)head + f.w;
                    int own = at >= 0 && at < p.num_free ? p.free_pages[at] : -1;
                    if (own >= p.num_pages) own = -1;
                    const int old = from[full];
                    if (own < 0 || old < 0 || old >= p.num_pages) bad = true;
                    else pair = make_int2(old, own);
                    if (lane == 0) to[full] = own;
                }
                if (lane == 0) __stcg(p.lens_out + f.y, f.z);
            }
            if (lane == 0) {
                p.pairs[2ll * (base + k)] = pair.x;
                p.pairs[2ll * (base + k) + 1] = pair.y;
            }
        }
        taken += total;
    }
    if (me == 0) p.head_out[0] = (int)max((long long)min(head, 0), min((long long)head + taken, (long long)max(head, p.num_free)));
    if (bad) set_status(p.status, STATUS_BAD_PAGE);
}

// ---- a CTA's share of the pages, PG_CHUNK at a time, in the order of their numbers ----
struct PageWalk {
    int first, last;                             // in whole eights
    uint32_t masks[PG_KEEP];
    int before[PG_KEEP];                         // pages in a mask before the thread's, among the CTA's
    int kept;                                    // and before the chunks that are not kept

    __device__ __forceinline__ explicit PageWalk(int num_pages) {
        const int each = (int)((((long long)num_pages + PG_CTAS - 1) / PG_CTAS + PG_PER - 1) / PG_PER * PG_PER);
        first = (int)min((long long)num_pages, (long long)cluster_rank() * each);
        last = (int)min((long long)num_pages, (long long)first + each);
    }
    // mask_of(first page, pages): their mask.  Returns how many of the CTA's pages are in one.
    template <typename MASK>
    __device__ __forceinline__ int scan(int* sums, MASK mask_of) {
        int running = 0, total;
#pragma unroll
        for (int c = 0; c < PG_KEEP; ++c) {
            const int at = first + c * PG_CHUNK + (int)threadIdx.x * PG_PER;
            masks[c] = 0u;
            if (first + c * PG_CHUNK < last) {
                if (at < last) masks[c] = mask_of(at, min(PG_PER, last - at));
                before[c] = running + block_before(__popc(masks[c]), total, sums);
                running += total;
            }
        }
        kept = running;
        for (int base = first + PG_KEEP * PG_CHUNK; base < last; base += PG_CHUNK) {
            const int at = base + (int)threadIdx.x * PG_PER;
            block_before(at < last ? __popc(mask_of(at, min(PG_PER, last - at))) : 0, total, sums);
            running += total;
        }
        return running;
    }
    // f(first page, pages, mask, pages in a mask before the first); mask_of has to give what it gave.
    template <typename MASK, typename FUNC>
    __device__ __forceinline__ void each(int* sums, MASK mask_of, FUNC f) const {
#pragma unroll
        for (int c = 0; c < PG_KEEP; ++c) {
            const int at = first + c * PG_CHUNK + (int)threadIdx.x * PG_PER;
            if (at < last) f(at, min(PG_PER, last - at), masks[c], before[c]);
        }
        int running = kept, total;
        for (int base = first + PG_KEEP * PG_CHUNK; base < last; base += PG_CHUNK) {
            const int at = base + (int)threadIdx.x * PG_PER;
            const uint32_t mask = at < last ? mask_of(at, min(PG_PER, last - at)) : 0u;
            const int ahead = running + block_before(__popc(mask), total, sums);
            if (at < last) f(at, min(PG_PER, last - at), mask, ahead);
            running += total;
        }
    }
};

// n of PG_PER words from an array on 16 bytes, `at` in whole eights; the others 0.
__device__ __forceinline__ void load_words(const int32_t* from, int at, int n, int (&x)[PG_PER]) {
    if (n == PG_PER) {
        const int4 a = __ldcg(reinterpret_cast<const int4*>(from + at)), b = __ldcg(reinterpret_cast<const int4*>(from + at) + 1);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
#pragma unroll
        for (int k = 0; k < PG_PER; ++k) x[k] = k < n ? __ldcg(from + at + k) : 0;
    }
}

// ---- free ----
// refs_out starts as the owners beside the first and loses one for each row
// that gives the page back, so it is negative where the last one has.
__global__ void __cluster_dims__(PG_CTAS, 1, 1) __launch_bounds__(PG_THREADS, 1) page_free_kernel(const __grid_constant__ PageParams p) {
    __shared__ int sums[PG_WARPS], slots[PG_CTAS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)cluster_rank(), me = rank * PG_THREADS + tid;
    const long long head = p.free_head[0];
    bool bad = false;
    if (me == 0 && p.status) __stcg(p.status, 0u);
    copy_words(p.refs, p.refs_out, p.num_pages, me, [](int x) { return max(x, 0); });
    cluster_barrier();
    // A warp takes up to 32 rows, a lane looks a row's lengths up; then the cells of all of them, a lane a cell.
    const int rows = min(32, max(1, (p.N + PG_ALL / 32 - 1) / (PG_ALL / 32)));
    for (int n0 = (rank * PG_WARPS + warp) * rows; n0 < p.N; n0 += PG_ALL / 32 * rows) {
        const int n = n0 + lane;
        int from = 0, cells = 0;
        if (lane < rows && n < p.N) {
            const int len = p.lens[n], keep = p.keep[n], kept = max(0, min(keep, len));
            bad |= keep != kept;
            from = row_pages(p, kept, bad);
            cells = row_pages(p, len, bad) - from;
            p.lens_out[n] = kept;
        }
        int upto = cells;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += y;
        }
        const int all = __shfl_sync(0xffffffffu, upto, 31);
        const int32_t* cell0 = p.table + (long long)n * p.width + from - (upto - cells);   // cell i of the warp's, if in this row
        for (int base = 0; base < all; base += 8 * 32) {
            int page[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int i = base + 32 * k + lane;
                int row = 0;                     // rows whose cells end at or before i
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) {
                    const int end = __shfl_sync(0xffffffffu, upto, row + d - 1);
                    if (end <= i) row += d;
                }
                const unsigned long long at = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(cell0), row & 31);
                page[k] = i < all ? __ldg(reinterpret_cast<const int32_t*>(at) + i) : 0;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (base + 32 * k + lane < all) {
                    if (page[k] >= 0 && page[k] < p.num_pages) atomicSub(p.refs_out + page[k], 1);
                    else bad = true;
                }
        }
    }
    cluster_barrier();
    PageWalk walk(p.num_pages);
    auto freed = [&](int at, int n) {
        int x[PG_PER];
        load_words(p.refs_out, at, n, x);
        uint32_t mask = 0;
#pragma unroll
        for (int k = 0; k < PG_PER; ++k)
            if (x[k] < 0) mask |= 1u << k, bad |= x[k] < -1;
        return mask;
    };
    const int mine = walk.scan(sums, freed);
    int all;
    const int before = cluster_before(mine, all, slots);
    walk.each(sums, freed, [&](int at, int, uint32_t mask, int ahead) {
        long long to = head - all + before + ahead;
        for (; mask != 0u; mask &= mask - 1, ++to) {
            const int page = at + __ffs(mask) - 1;
            p.refs_out[page] = 0;
            if (to >= 0 && to < p.num_free) p.free_io[to] = page;
            else bad = true;
        }
    });
    if (me == 0) p.head_out[0] = (int)max(0ll, head - all);
    if (bad) set_status(p.status, STATUS_BAD_PAGE);
}

// ---- compact ----
// `moved` marks the free pages until it is written.
__global__ void __cluster_dims__(PG_CTAS, 1, 1) __launch_bounds__(PG_THREADS, 1) page_compact_kernel(const __grid_constant__ PageParams p) {
    __shared__ int sums[PG_WARPS], slots[2][PG_CTAS];
    const int rank = (int)cluster_rank(), me = rank * PG_THREADS + (int)threadIdx.x;
    const long long head = p.free_head[0];
    bool bad = false;
    if (me == 0 && p.status) __stcg(p.status, 0u);
    fill_words(p.moved, 0, p.num_pages, me);
    cluster_barrier();
    for (long long i = max(head, 0ll) + me; i < p.num_free; i += PG_ALL) {
        const int page = p.free_pages[i];
        if (page < 0 || page >= p.num_pages || atomicExch(p.moved + page, 1) != 0) bad = true;
    }
    cluster_barrier();
    PageWalk walk(p.num_pages);
    auto is_free = [&](int at, int n) {
        int x[PG_PER];
        load_words(p.moved, at, n, x);
        uint32_t mask = 0;
#pragma unroll
        for (int k = 0; k < PG_PER; ++k)
            if (x[k] != 0) mask |= 1u << k;
        return mask;
    };
    int all, holes, total;
    const int mine = walk.scan(sums, is_free), before = cluster_before(mine, all, slots[0]), used = p.num_pages - all;
    int below = 0;                               // free pages below `used`
    walk.each(sums, is_free, [&](int at, int n, uint32_t mask, int) {
        below += __popc(mask & (used - at >= PG_PER ? 0xffu : used > at ? (1u << (used - at)) - 1 : 0u));
    });
    block_before(below, total, sums);
    cluster_before(total, holes, slots[1]);
    // the k-th free page below `used` takes the k-th used one from there on
    auto place = [&](auto f) {
        walk.each(sums, is_free, [&](int at, int n, uint32_t mask, int ahead) {
            int free_before = before + ahead;
#pragma unroll
            for (int k = 0; k < PG_PER; ++k)
                if (k < n) {
                    const int i = at + k;
                    const bool hole = (mask >> k) & 1u;
                    f(i, hole, hole ? free_before : (i - used) - (free_before - holes));
                    free_before += hole;
                }
        });
    };
    place([&](int i, bool hole, int k) {
        if (hole == (i < used)) __stcg(p.pairs + 2ll * k + (hole ? 1 : 0), i);
    });
    for (int i = 2 * holes + me; i < p.num_pages / 2 * 2; i += PG_ALL) p.pairs[i] = -1;
    cluster_barrier();
    place([&](int i, bool hole, int k) {
        int to = i;
        if (hole) to = -1;
        else if (i >= used) to = __ldcg(p.pairs + 2ll * k + 1);
        p.moved[i] = to;
        if (to >= 0) p.refs_out[to] = __ldg(p.refs + i);
        if (i >= used) p.refs_out[i] = 0;
    });
    for (int i = me; i < p.num_free; i += PG_ALL) {
        const long long to = used + (i - head);
        p.free_out[i] = i < head ? p.free_pages[i] : to < p.num_pages ? (int)to : -1;
    }
    if (me == 0) p.count[0] = holes;
    if (bad) set_status(p.status, STATUS_BAD_PAGE);
}

// The table's cells, by their pages' new numbers.
__global__ void __launch_bounds__(256) page_remap_kernel(const __grid_constant__ PageParams p, int32_t* out) {
    const long long cells = (long long)p.N * p.width;
    bool bad = false;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < cells; i += (long long)gridDim.x * 256) {
        const int n = (int)(i / p.width), col = (int)(i - (long long)n * p.width);
        int to = -1;
        if (col < row_pages(p, p.lens[n], bad)) {
            const int page = p.table[i];
            if (page >= 0 && page < p.num_pages) to = p.moved[page];
            bad |= to < 0;
        }
        out[i] = to;
    }
    if (bad) set_status(p.status, STATUS_BAD_PAGE);
}

// ---- copy: pieces of up to 32 KiB of all pairs and pools, dealt to the CTAs ----
constexpr int COPY_POOLS = 64;                   // of one launch
constexpr int COPY_THREADS = 256;
constexpr int COPY_PER = 8;                      // 16-byte words of a thread

struct CopyParams {
    uint4* pools[COPY_POOLS];
    const int32_t* pairs;
    const int32_t* count;
    uint32_t* status;
    long long words;                             // of a page
    long long pieces;
    int piece;                                   // words of one
    int num_pools, num_pages, F;
};

__global__ void __launch_bounds__(COPY_THREADS) page_copy_kernel(const __grid_constant__ CopyParams p) {
    const int pairs = p.count ? max(0, min(p.F, p.count[0])) : p.F;
    const long long each = p.pieces * p.num_pools, items = each * pairs;
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        const long long pair = item / each, rest = item - pair * each;
        const long long pool = rest / p.pieces, first = (rest - pool * p.pieces) * p.piece;
        const int src = p.pairs[2 * pair], dst = p.pairs[2 * pair + 1];
        if (src < 0 || dst < 0) continue;
        if (src >= p.num_pages || dst >= p.num_pages) {
            if (threadIdx.x == 0) set_status(p.status, STATUS_BAD_PAGE);
            continue;
        }
        const int count = (int)min((long long)p.piece, p.words - first);
        const uint4* from = p.pools[pool] + src * p.words + first;
        uint4* to = p.pools[pool] + dst * p.words + first;
        uint4 x[COPY_PER];
#pragma unroll
        for (int k = 0; k < COPY_PER; ++k) {
            const int at = threadIdx.x + COPY_THREADS * k;
            if (at < count) x[k] = __ldcs(from + at);
        }
#pragma unroll
        for (int k = 0; k < COPY_PER; ++k) {
            const int at = threadIdx.x + COPY_THREADS * k;
            if (at < count) __stcs(to + at, x[k]);
        }
    }
}

bool off(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

template <typename... P>
bool missing(const P*... p) { return ((p == nullptr) || ...); }
template <typename... P>
bool off4(const P*... p) { return (off(p, 4) || ...); }

// What the three share: sizes, the table, the free list, the status header.
bool common_ok(const PageParams& p, const void* table) {
    if (p.N < 1 || p.width < 0 || p.num_pages < 1 || p.num_free < 0 || p.page_size < 1) return false;
    if ((p.width > 0 && !table) || missing(p.lens, p.refs, p.refs_out, p.free_head)) return false;
    return !off4(table, p.lens, p.refs, p.free_head) && !off(p.refs_out, 16) && !off(p.status, 256);
}

kda_status launched() { return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace

}  // namespace kda

extern "C" {


kda_status kda_page_fork(int32_t* block_table, int table_width, const int32_t* seq_lens, const int32_t* parents,
                         const int32_t* children, const int32_t* refs, int num_pages, const int32_t* free_pages,
                         int num_free, const int32_t* free_head, int page_size, int32_t* seq_lens_out,
                         int32_t* refs_out, int32_t* free_head_out, int32_t* pairs, int N, int F, void* workspace,
                         cudaStream_t stream) {
    using namespace kda;
    PageParams p{};
    p.status = static_cast<uint32_t*>(workspace);
    p.table_io = block_table, p.lens = seq_lens, p.parents = parents, p.children = children, p.refs = refs;
    p.free_pages = free_pages, p.free_head = free_head, p.lens_out = seq_lens_out, p.refs_out = refs_out;
    p.head_out = free_head_out, p.pairs = pairs;
    p.width = table_width, p.num_pages = num_pages, p.num_free = num_free, p.page_size = page_size, p.N = N, p.F = F;
    if (!common_ok(p, block_table) || F < 0) return KDA_ERR_INVALID_ARG;
    if (missing(seq_lens_out, free_head_out) || (F > 0 && missing(parents, children, pairs)) || (num_free > 0 && !free_pages))
        return KDA_ERR_INVALID_ARG;
    if (off4(parents, children, free_pages, seq_lens_out, free_head_out, pairs)) return KDA_ERR_INVALID_ARG;
    page_fork_kernel<<<PG_CTAS, PG_THREADS, 0, stream>>>(p);
    return launched();
}

kda_status kda_page_copy(void* const* pools, int num_pools, int num_pages, long long page_bytes, const int32_t* pairs,
                         const int32_t* count, int F, void* workspace, cudaStream_t stream) {
    using namespace kda;
    if (num_pools < 1 || !pools || num_pages < 1 || F < 0 || page_bytes < 16 || page_bytes % 16 != 0 || page_bytes >= (1ll << 40))
        return KDA_ERR_INVALID_ARG;
    if ((F > 0 && !pairs) || off4(pairs, count) || off(workspace, 256)) return KDA_ERR_INVALID_ARG;
    for (int i = 0; i < num_pools; ++i)
        if (!pools[i] || off(pools[i], 16)) return KDA_ERR_INVALID_ARG;
    CopyParams p{};
    p.pairs = pairs, p.count = count, p.status = static_cast<uint32_t*>(workspace), p.words = page_bytes / 16;
    p.num_pages = num_pages, p.F = F;
    const long long most_words = COPY_THREADS * COPY_PER;
    p.pieces = (p.words + most_words - 1) / most_words;   // equal ones
    p.piece = (int)((p.words + p.pieces - 1) / p.pieces);
    if (p.status && cudaMemsetAsync(p.status, 0, WS_CLEAR, stream) != cudaSuccess) return KDA_ERR_CUDA;
    if (F == 0) return KDA_OK;
    for (int first = 0; first < num_pools; first += COPY_POOLS) {
        p.num_pools = num_pools - first < COPY_POOLS ? num_pools - first : COPY_POOLS;
        for (int i = 0; i < p.num_pools; ++i) p.pools[i] = static_cast<uint4*>(pools[first + i]);
        const long long items = p.pieces * p.num_pools * F, most = 152ll * 8;
        page_copy_kernel<<<(unsigned)(items < most ? items : most), COPY_THREADS, 0, stream>>>(p);
        if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
    }
    return KDA_OK;
}

kda_status kda_page_free(const int32_t* block_table, int table_width, const int32_t* seq_lens,
                         const int32_t* keep_lens, const int32_t* refs, int num_pages, int32_t* free_pages,
                         int num_free, const int32_t* free_head, int page_size, int32_t* seq_lens_out,
                         int32_t* refs_out, int32_t* free_head_out, int N, void* workspace, cudaStream_t stream) {
    using namespace kda;
    PageParams p{};
    p.status = static_cast<uint32_t*>(workspace);
    p.table = block_table, p.lens = seq_lens, p.keep = keep_lens, p.refs = refs, p.free_io = free_pages;
    p.free_head = free_head, p.lens_out = seq_lens_out, p.refs_out = refs_out, p.head_out = free_head_out;
    p.width = table_width, p.num_pages = num_pages, p.num_free = num_free, p.page_size = page_size, p.N = N;
    if (!common_ok(p, block_table)) return KDA_ERR_INVALID_ARG;
    if (missing(keep_lens, seq_lens_out, free_head_out) || (num_free > 0 && !free_pages)) return KDA_ERR_INVALID_ARG;
    if (off4(keep_lens, free_pages, seq_lens_out, free_head_out)) return KDA_ERR_INVALID_ARG;
    page_free_kernel<<<PG_CTAS, PG_THREADS, 0, stream>>>(p);
    return launched();
}

kda_status kda_page_compact(const int32_t* block_table, int table_width, const int32_t* seq_lens, const int32_t* refs,
                            int num_pages, const int32_t* free_pages, int num_free, const int32_t* free_head,
                            int page_size, int32_t* table_out, int32_t* refs_out, int32_t* free_out, int32_t* pairs,
                            int32_t* count, int32_t* moved, int N, void* workspace, cudaStream_t stream) {
    using namespace kda;
    PageParams p{};
    p.status = static_cast<uint32_t*>(workspace);
    p.table = block_table, p.lens = seq_lens, p.refs = refs, p.free_pages = free_pages, p.free_head = free_head;
    p.refs_out = refs_out, p.free_out = free_out, p.pairs = pairs, p.count = count, p.moved = moved;
    p.width = table_width, p.num_pages = num_pages, p.num_free = num_free, p.page_size = page_size, p.N = N;
    if (!common_ok(p, block_table)) return KDA_ERR_INVALID_ARG;
    if (missing(count, moved) || (num_free > 0 && missing(free_pages, free_out)) || (num_pages > 1 && !pairs) ||
        (table_width > 0 && !table_out))
        return KDA_ERR_INVALID_ARG;
    if (off4(free_pages, free_out, pairs, count, table_out) || off(moved, 16)) return KDA_ERR_INVALID_ARG;
    page_compact_kernel<<<PG_CTAS, PG_THREADS, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
    const long long blocks = ((long long)N * table_width + 255) / 256, most = 152ll * 8;
    if (blocks == 0) return KDA_OK;
    page_remap_kernel<<<(unsigned)(blocks < most ? blocks : most), 256, 0, stream>>>(p, table_out);
    return launched();
}

}  // extern "C"
