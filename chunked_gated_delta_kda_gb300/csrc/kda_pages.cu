// Pages that several requests own: forking, freeing, compacting and copying
// (kda_page_fork, kda_page_free, kda_page_compact, kda_page_copy), with their
// C entry points.  See include/kda.h for the contract.
//
// The first three are bookkeeping of a few thousand words whose steps depend
// on each other (owners counted before pages are given back), so latency
// bounds them, and a step between CTAs is what costs.  Forking and freeing run
// as one cluster of eight CTAs with cluster barriers between the steps: one
// launch and no scratch memory, the outputs hold what the steps pass on, and
// what one CTA writes and another reads goes through the L2 (atomics, __stcg,
// __ldcg).  Compacting needs no steps (see there).  Measured, in a graph: 256
// forks of up to 128 pages 8 us, 8 forks 5; 256 requests that go back by up
// to seven tokens 8.6; 2048 that end or stay, 100 thousand cells, 17.5; 512
// pages compacted in 4.3, 8192 in 6.0, a million in 121 (each CTA reads the
// whole free list, through the L2).  Copying pages is bound by HBM: 297 MB each
// way 91 us, 6.5 TB/s, 96 % of what a plain copy reaches.
#include <cstdint>

#include "kda.h"
#include "kda_latent_mma.cuh"

namespace kda {

namespace {

constexpr int PG_CTAS = 8;
constexpr int PG_THREADS = 1024;
constexpr int PG_WARPS = PG_THREADS / 32;
constexpr int PG_ALL = PG_CTAS * PG_THREADS;
constexpr int PG_SHARES = PG_CTAS * PG_WARPS;    // the cluster's warps, each with a share of the pages
constexpr long long FREE_ALONE = 1 << 17;        // cells that the cluster gives back by itself
constexpr int PG_MOST = 1 << 30;                 // rows, columns, pages, entries: an index that steps past them stays in 32 bits

struct PageParams {
    const int32_t* table;
    int32_t* table_io;
    const int32_t* lens;
    const int32_t* keep;
    const int32_t* parents;
    const int32_t* children;
    const int32_t* fork_lens;
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
__device__ __forceinline__ void copy_words(const int32_t* from, int32_t* to, int count, int me, FUNC f, int all = PG_ALL) {
    if (((reinterpret_cast<uintptr_t>(from) | reinterpret_cast<uintptr_t>(to)) & 15u) == 0) {
        const int quads = count >> 2;
#pragma unroll 4
        for (int i = me; i < quads; i += all) {
            const int4 x = __ldg(reinterpret_cast<const int4*>(from) + i);
            __stcg(reinterpret_cast<int4*>(to) + i, make_int4(f(x.x), f(x.y), f(x.z), f(x.w)));
        }
        if (me < (count & 3)) __stcg(to + 4 * quads + me, f(__ldg(from + 4 * quads + me)));
        return;
    }
#pragma unroll 4
    for (int i = me; i < count; i += all) __stcg(to + i, f(__ldg(from + i)));
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

// ---- fork: a warp an entry ----
// Up to 256 entries (FEW) every CTA looks for earlier entries with the same
// child in its shared memory; beyond, entries claim their children: lens_out
// holds i - F at a child of length 0 that entry i is the first to have. That
// takes two barriers more, the search a time that grows with the entries:
// forks of a page 4.1 us by search and 5.1 by claims for 8, 5.3 and 6.0 for
// 256, 7.7 and 7.0 for 512, 14.7 and 8.7 for 1024.
constexpr int PG_FEW = 256;

template <bool FEW>
__global__ void __cluster_dims__(PG_CTAS, 1, 1) __launch_bounds__(PG_THREADS, 1) page_fork_kernel(const __grid_constant__ PageParams p) {
    __shared__ int sums[PG_WARPS];
    __shared__ int4 wanted[FEW ? PG_FEW / 4 : 1];   // the children of entries that may have them, else -1
    __shared__ int4 entries[PG_THREADS];         // parent (-1: skipped), child, tokens, place among the own pages (-1: none)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)cluster_rank(), me = rank * PG_THREADS + tid;
    const int head = p.free_head[0];
    bool bad = false;
    if (me == 0 && p.status) __stcg(p.status, 0u);
    auto same = [](int x) { return x; };
    copy_words(p.refs, p.refs_out, p.num_pages, me, same);
    copy_words(p.lens, p.lens_out, p.N, me, same);
    auto may_have = [&](int a, int c) { return c >= 0 && c < p.N && a >= 0 && a < p.N && p.lens[c] == 0; };
    if constexpr (FEW) {
        if (tid < PG_FEW) reinterpret_cast<int*>(wanted)[tid] = tid < p.F && may_have(p.parents[tid], p.children[tid]) ? p.children[tid] : -1;
        __syncthreads();
    } else {
        cluster_barrier();
        for (int i = me; i < p.F; i += PG_ALL) {
            const int a = p.parents[i], c = p.children[i];
            if (may_have(a, c)) atomicMin(p.lens_out + c, i - p.F);
        }
        cluster_barrier();
    }
    int taken = 0;
    for (int base = 0; base < p.F; base += PG_THREADS) {
        const int i = base + tid;
        int4 e = make_int4(-1, -1, 0, -1);
        if (i < p.F) {
            const int a = p.parents[i], c = p.children[i];
            if (c >= 0) {
                bool first = may_have(a, c);
                if constexpr (FEW) {
                    for (int k = 0; k < tid / 4; ++k) {
                        const int4 w = wanted[k];
                        if (w.x == c || w.y == c || w.z == c || w.w == c) first = false;
                    }
                    for (int k = tid / 4 * 4; k < tid; ++k)
                        if (reinterpret_cast<const int*>(wanted)[k] == c) first = false;
                } else if (first) {
                    first = __ldcg(p.lens_out + c) == i - p.F;
                }
                if (first) {
                    const long long most = (long long)p.width * p.page_size;
                    const int len = p.lens[a], whole = (int)max(0ll, min((long long)len, most));
                    const int taken_over = p.fork_lens ? p.fork_lens[i] : whole, some = max(0, min(taken_over, whole));
                    bad |= len != whole || taken_over != some;
                    e = make_int4(a, c, some, -1);
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
        cluster_barrier();                       // the copies are there, and every CTA has looked its entries up
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
                    if (own < 0 || own >= p.num_pages) own = -1;
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

// ---- the pages in the order of their numbers, a share a warp ----
struct Share {
    int first, last;                             // in whole lines of 128 pages
    __device__ __forceinline__ Share(int num_pages, int index) {
        const int each = (int)((((long long)num_pages + PG_SHARES - 1) / PG_SHARES + 127) / 128 * 128);
        first = (int)min((long long)num_pages, (long long)index * each);
        last = (int)min((long long)num_pages, (long long)first + each);
    }
};

// Whole warp: f(first page of the lane, its four words of `from` (on 16 bytes), how many of them there are), 128 pages a time.
template <typename FUNC>
__device__ __forceinline__ void walk(const int32_t* from, int first, int last, FUNC f) {
    const int lane = threadIdx.x & 31;
    for (int base = first; base < last; base += 4 * 128) {
        int x[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int at = base + 128 * u + 4 * lane;
            if (at + 4 <= last) {
                const int4 v = __ldcg(reinterpret_cast<const int4*>(from + at));
                x[u][0] = v.x, x[u][1] = v.y, x[u][2] = v.z, x[u][3] = v.w;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) x[u][k] = at + k < last ? __ldcg(from + at + k) : 0;
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (base + 128 * u < last) {
                const int at = base + 128 * u + 4 * lane;
                f(at, x[u], max(0, min(4, last - at)));
            }
    }
}

// How many of the pages that are marked (mark(word)) come before the lane's, among the warp's 128 ones; all of them in `total`.
template <typename MARK>
__device__ __forceinline__ int lanes_before(const int (&x)[4], int n, MARK mark, int& total) {
    const uint32_t lower = (1u << (threadIdx.x & 31)) - 1;
    int before = 0;
    total = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t marked = __ballot_sync(0xffffffffu, k < n && mark(x[k]));
        before += __popc(marked & lower);
        total += __popc(marked);
    }
    return before;
}

// Every warp's number to all CTAs of the cluster, and back: the sum of those of the shares before `index`, and of all
// where index is PG_SHARES.  Between the two, a cluster barrier.
__device__ __forceinline__ void send_count(int mine, int index, int* counts) {
    const int lane = threadIdx.x & 31;
    if (lane < PG_CTAS) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(smem_u32(counts + index), lane)), "r"(mine) : "memory");
}
__device__ __forceinline__ int shares_before(int index, const int* counts) {
    int sum = 0;
#pragma unroll
    for (int k = 0; k < PG_SHARES; k += 32) {
        const int i = k + (int)(threadIdx.x & 31);
        if (i < index) sum += counts[i];
    }
    return __reduce_add_sync(0xffffffffu, sum);
}

// ---- free ----
// refs_out starts as the owners beside the first and loses one for each row
// that gives the page back, so it is negative where the last one has.

// A warp takes `rows` rows at a time, a lane looks a row's lengths up; then the cells of all of them, a lane a cell.
__device__ __forceinline__ void release_rows(const PageParams& p, int warp, int warps, int rows, bool& bad) {
    const int lane = threadIdx.x & 31;
    for (long long n0 = (long long)warp * rows; n0 < p.N; n0 += (long long)warps * rows) {
        const int n = (int)n0 + lane;
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
}

__device__ __forceinline__ int owners(int refs) { return max(refs, 0); }

// Where many cells may be given back, the whole GPU does that, in two kernels in front of the cluster, whose eight SMs
// take about a cell a clock each.  How many are given back only the device knows.  The limit, of the table's cells, is
// where a step of drafts breaks even, which gives back few; where requests end it would be lower.  Rows of 512 cells, us
// a call, by the cluster alone / so: a step that takes back up to seven tokens 64 rows 7.1 / 10, 128 7.8 / 10, 256
// 9.9 / 9.9, 512 13.3 / 11.8, 2048 32.5 / 24.8; two in three rows ended 64 16.6 / 12.2, 128 18.5 / 13.8, 256 23.3 / 18.7,
// 512 38.7 / 26.4, 2048 126 / 77 (two more launches are 5 us on the host).
__global__ void __launch_bounds__(256) page_owners_kernel(const __grid_constant__ PageParams p) {
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
    const int me = blockIdx.x * 256 + threadIdx.x;
    if (me == 0 && p.status) *p.status = 0u;
    copy_words(p.refs, p.refs_out, p.num_pages, me, owners, gridDim.x * 256);
}
__global__ void __launch_bounds__(256) page_release_kernel(const __grid_constant__ PageParams p, int rows) {
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
    bool bad = false;
    release_rows(p, blockIdx.x * 8 + (threadIdx.x >> 5), gridDim.x * 8, rows, bad);
    if (bad) set_status(p.status, STATUS_BAD_PAGE);
}

template <bool ALONE>
__global__ void __cluster_dims__(PG_CTAS, 1, 1) __launch_bounds__(PG_THREADS, 1) page_free_kernel(const __grid_constant__ PageParams p) {
    __shared__ int counts[PG_SHARES];
    const int rank = (int)cluster_rank(), me = rank * PG_THREADS + (int)threadIdx.x, index = me >> 5;
    if constexpr (ALONE) asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
    else asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    bool bad = false;
    if constexpr (ALONE) {
        if (me == 0 && p.status) __stcg(p.status, 0u);
        copy_words(p.refs, p.refs_out, p.num_pages, me, owners);
        cluster_barrier();
        release_rows(p, index, PG_SHARES, min(32, max(1, (p.N + PG_SHARES - 1) / PG_SHARES)), bad);
        cluster_barrier();
    } else {
        cluster_barrier();                       // the other CTAs' shared memory is there
        asm volatile("griddepcontrol.wait;" ::: "memory");
    }
    const long long head = p.free_head[0];
    // rows that go back into a page with another owner left
    for (int n = me; n < p.N; n += PG_ALL) {
        const int len = p.lens[n], kept = max(0, min(p.keep[n], len));
        if (kept < len && kept % p.page_size != 0 && kept / p.page_size < p.width) {
            const int page = p.table[(long long)n * p.width + kept / p.page_size];
            bad |= page < 0 || page >= p.num_pages || __ldcg(p.refs_out + page) > 0;
        }
    }
    const Share share(p.num_pages, index);
    int mine = 0;
    walk(p.refs_out, share.first, share.last, [&](int, const int(&x)[4], int) {
#pragma unroll
        for (int k = 0; k < 4; ++k) mine += x[k] < 0, bad |= x[k] < -1;
    });
    send_count(__reduce_add_sync(0xffffffffu, mine), index, counts);
    cluster_barrier();
    const int all = shares_before(PG_SHARES, counts);
    long long to = head - all + shares_before(index, counts);
    walk(p.refs_out, share.first, share.last, [&](int at, const int(&x)[4], int n) {
        int total;
        long long place = to + lanes_before(x, n, [](int v) { return v < 0; }, total);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (x[k] < 0) {
                p.refs_out[at + k] = 0;
                if (place >= 0 && place < p.num_free) p.free_io[place] = at + k;
                else bad = true;
                ++place;
            }
        to += total;
    });
    if (me == 0) p.head_out[0] = (int)max(0ll, head - all);
    if (bad) set_status(p.status, STATUS_BAD_PAGE);
}

// ---- compact ----
// Every CTA marks the free pages as bits in its shared memory, all of them, and
// counts them group by group.  So it knows each page's new number by itself
// (the k-th used page from `used` on, the number of used ones, goes to the k-th
// free one below, found by bisection) and takes its share of the pages, of the
// free list and of the table, with no step between the CTAs.
constexpr int CP_GROUP = 256;                    // pages of a count
constexpr int CP_GROUP_BYTES = CP_GROUP / 8 + 4; // bits and count
constexpr int CP_MOST = 1 << 20;                 // pages; as bits 128 KiB

struct FreePages {
    const uint32_t* bits;
    const int* counts;                           // free pages before each group
    int groups, used, holes;                     // holes: free pages below `used`
    __device__ __forceinline__ bool is_free(int page) const { return (bits[page >> 5] >> (page & 31)) & 1u; }
    __device__ __forceinline__ int before(int page) const {
        int n = counts[page / CP_GROUP];
        for (int w = page / CP_GROUP * (CP_GROUP / 32); w < page >> 5; ++w) n += __popc(bits[w]);
        return n + __popc(bits[page >> 5] & ((1u << (page & 31)) - 1));
    }
    __device__ __forceinline__ int select(int k) const {
        int lo = 0, hi = groups - 1;             // the last group with at most k before it
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (counts[mid] <= k) lo = mid;
            else hi = mid - 1;
        }
        k -= counts[lo];
        int w = lo * (CP_GROUP / 32);
        for (int c; (c = __popc(bits[w])) <= k; ++w) k -= c;
        uint32_t word = bits[w];
        for (; k > 0; --k) word &= word - 1;
        return 32 * w + __ffs(word) - 1;
    }
    // The page's new number, -1 for a free one; k: its place among those that move, or -1.
    __device__ __forceinline__ int moved(int page, int& k) const {
        k = -1;
        if (is_free(page)) return -1;
        if (page < used) return page;
        k = (page - used) - (before(page) - holes);
        return select(k);
    }
};

__global__ void __launch_bounds__(PG_THREADS, 1) page_compact_kernel(const __grid_constant__ PageParams p, int32_t* table_out) {
    extern __shared__ uint32_t bits[];           // of whole groups, then the counts
    __shared__ int sums[PG_WARPS];
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, groups = (p.num_pages + CP_GROUP - 1) / CP_GROUP, words = groups * (CP_GROUP / 32);
    int* counts = reinterpret_cast<int*>(bits + words);
    const long long head = p.free_head[0];
    bool bad = false;
    for (int i = tid; i < words; i += PG_THREADS) bits[i] = 0u;
    __syncthreads();
#pragma unroll 8
    for (long long i = max(head, 0ll) + tid; i < p.num_free; i += PG_THREADS) {
        const int page = __ldg(p.free_pages + i);
        if (page < 0 || page >= p.num_pages || ((atomicOr(bits + (page >> 5), 1u << (page & 31)) >> (page & 31)) & 1u) != 0u) bad = true;
    }
    __syncthreads();
    int all = 0;
    for (int base = 0; base < groups; base += PG_THREADS) {
        const int g = base + tid;
        int mine = 0, total;
        if (g < groups)
#pragma unroll
            for (int w = 0; w < CP_GROUP / 32; ++w) mine += __popc(bits[g * (CP_GROUP / 32) + w]);
        const int before = block_before(mine, total, sums);
        if (g < groups) counts[g] = all + before;
        all += total;
    }
    __syncthreads();
    FreePages f{bits, counts, groups, p.num_pages - all, all};
    if (f.used < p.num_pages) f.holes = f.before(f.used);

    const int me = blockIdx.x * PG_THREADS + tid, threads = gridDim.x * PG_THREADS;
    int k;
    for (int i = me; i < p.num_pages; i += threads) {
        const int to = f.moved(i, k);
        p.moved[i] = to;
        if (to >= 0) p.refs_out[to] = __ldg(p.refs + i);
        if (i >= f.used) p.refs_out[i] = 0;
        if (k >= 0) p.pairs[2ll * k] = i, p.pairs[2ll * k + 1] = to;
    }
    for (int i = 2 * f.holes + me; i < p.num_pages / 2 * 2; i += threads) p.pairs[i] = -1;
    for (int i = me; i < p.num_free; i += threads) {
        const long long to = f.used + (i - head);
        p.free_out[i] = i < head ? __ldg(p.free_pages + i) : to < p.num_pages ? (int)to : -1;
    }
    const long long cells = (long long)p.N * p.width;
    for (long long i = me; i < cells; i += threads) {
        const int n = (int)(i / p.width), col = (int)(i - (long long)n * p.width);
        int to = -1;
        if (col < row_pages(p, p.lens[n], bad)) {
            const int page = __ldg(p.table + i);
            if (page >= 0 && page < p.num_pages) to = f.moved(page, k);
            bad |= to < 0;
        }
        table_out[i] = to;
    }
    if (me == 0) p.count[0] = f.holes;
    if (bad) set_status(p.status, STATUS_BAD_PAGE);
}

// More pages than fit as bits: through memory, in steps of one cluster, and the table behind it.  `moved` marks the free
// pages until it is written.
__global__ void __cluster_dims__(PG_CTAS, 1, 1) __launch_bounds__(PG_THREADS, 1) page_compact_large_kernel(const __grid_constant__ PageParams p) {
    __shared__ int counts[PG_SHARES], sums[PG_WARPS];
    const int rank = (int)cluster_rank(), me = rank * PG_THREADS + (int)threadIdx.x, index = me >> 5, warp = (int)threadIdx.x >> 5;
    const long long head = p.free_head[0];
    bool bad = false;
    fill_words(p.moved, 0, p.num_pages, me);
    cluster_barrier();
#pragma unroll 4
    for (long long i = max(head, 0ll) + me; i < p.num_free; i += PG_ALL) {
        const int page = p.free_pages[i];
        if (page < 0 || page >= p.num_pages || atomicExch(p.moved + page, 1) != 0) bad = true;
    }
    cluster_barrier();
    auto is_free = [](int v) { return v != 0; };
    const Share share(p.num_pages, index);
    auto count = [&](int first, int last) {
        int mine = 0;
        walk(p.moved, first, last, [&](int, const int(&x)[4], int) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mine += x[k] != 0;
        });
        return __reduce_add_sync(0xffffffffu, mine);
    };
    send_count(count(share.first, share.last), index, counts);
    cluster_barrier();
    const int used = p.num_pages - shares_before(PG_SHARES, counts);
    // free pages below `used`: those of the shares before the one that it is in, and of that up to there (a part a warp)
    const int each = max(128, Share(p.num_pages, 0).last), cut = min(PG_SHARES, used / each);
    const int part = (each / 128 + PG_WARPS - 1) / PG_WARPS * 128, first = min(used, cut * each + warp * part);
    const int some = count(first, min(used, first + part));
    if ((threadIdx.x & 31) == 0) sums[warp] = some;
    cluster_barrier();                           // (the marks are read for the last time but by their own share's warp)
    const int holes = shares_before(cut, counts) + __reduce_add_sync(0xffffffffu, sums[threadIdx.x & 31]);
    // The k-th free page below `used` takes the k-th used one from there on; `ahead`: free pages before the lane's.
    int ahead = shares_before(index, counts);
    walk(p.moved, share.first, share.last, [&](int at, const int(&x)[4], int n) {
        int total, before = ahead + lanes_before(x, n, is_free, total);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < n) {
                const int i = at + k;
                const bool hole = x[k] != 0, below = i < used;
                if (hole && below) p.pairs[2ll * before + 1] = i;
                if (!hole && !below) p.pairs[2ll * ((i - used) - (before - holes))] = i;
                if (hole || below) __stcg(p.moved + i, hole ? -1 : i);
                if (!below) __stcg(p.refs_out + i, 0);
                else if (!hole) p.refs_out[i] = __ldg(p.refs + i);
                before += hole;
            }
        ahead += total;
    });
    for (int i = 2 * holes + me; i < p.num_pages / 2 * 2; i += PG_ALL) p.pairs[i] = -1;
    for (int i = me; i < p.num_free; i += PG_ALL) {
        const long long to = used + (i - head);
        p.free_out[i] = i < head ? p.free_pages[i] : to < p.num_pages ? (int)to : -1;
    }
    if (me == 0) p.count[0] = holes;
    cluster_barrier();
    for (int k = me; k < holes; k += PG_ALL) {
        const int src = __ldcg(p.pairs + 2ll * k), dst = __ldcg(p.pairs + 2ll * k + 1);
        p.moved[src] = dst;
        p.refs_out[dst] = __ldg(p.refs + src);
    }
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
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
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
    if (p.N > PG_MOST || p.width > PG_MOST || p.num_pages > PG_MOST || p.num_free > PG_MOST) return false;
    if ((p.width > 0 && !table) || missing(p.lens, p.refs, p.refs_out, p.free_head)) return false;
    return !off4(table, p.lens, p.refs, p.free_head) && !off(p.refs_out, 16) && !off(p.status, 256);
}

// A kernel that may be set up while the one before it runs; it waits for that one itself.
template <typename... A, typename... B>
kda_status launch_early(void (*kernel)(A...), dim3 grid, int threads, int smem, cudaStream_t stream, const B&... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return succeeded(cudaLaunchKernelEx(&cfg, kernel, args...)) ? KDA_OK : KDA_ERR_CUDA;
}

// One that begins behind it.
template <typename... A>
kda_status launch(void (*kernel)(A...), dim3 grid, int threads, cudaStream_t stream, A... args) {
    void* at[] = {&args...};
    return succeeded(cudaLaunchKernel(kernel, grid, dim3((unsigned)threads), at, 0, stream)) ? KDA_OK : KDA_ERR_CUDA;
}

}  // namespace

}  // namespace kda

extern "C" {


kda_status kda_page_fork(int32_t* block_table, int table_width, const int32_t* seq_lens, const int32_t* parents,
                         const int32_t* children, const int32_t* fork_lens, const int32_t* refs, int num_pages,
                         const int32_t* free_pages, int num_free, const int32_t* free_head, int page_size,
                         int32_t* seq_lens_out, int32_t* refs_out, int32_t* free_head_out, int32_t* pairs, int N,
                         int F, void* workspace, cudaStream_t stream) {
    using namespace kda;
    PageParams p{};
    p.status = static_cast<uint32_t*>(workspace);
    p.table_io = block_table, p.lens = seq_lens, p.parents = parents, p.children = children, p.fork_lens = fork_lens, p.refs = refs;
    p.free_pages = free_pages, p.free_head = free_head, p.lens_out = seq_lens_out, p.refs_out = refs_out;
    p.head_out = free_head_out, p.pairs = pairs;
    p.width = table_width, p.num_pages = num_pages, p.num_free = num_free, p.page_size = page_size, p.N = N, p.F = F;
    if (!common_ok(p, block_table) || F < 0 || F > PG_MOST) return KDA_ERR_INVALID_ARG;
    if (missing(seq_lens_out, free_head_out) || (F > 0 && missing(parents, children, pairs)) || (num_free > 0 && !free_pages))
        return KDA_ERR_INVALID_ARG;
    if (off4(parents, children, fork_lens, free_pages, seq_lens_out, free_head_out, pairs)) return KDA_ERR_INVALID_ARG;
    // (an early launch is 1.2 us dearer on the host, which is what a fork of a few requests waits for)
    return launch(F <= PG_FEW ? page_fork_kernel<true> : page_fork_kernel<false>, dim3(PG_CTAS), PG_THREADS, stream, p);
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
    if (p.status && !succeeded(cudaMemsetAsync(p.status, 0, WS_CLEAR, stream))) return KDA_ERR_CUDA;
    if (F == 0) return KDA_OK;
    for (int first = 0; first < num_pools; first += COPY_POOLS) {
        p.num_pools = num_pools - first < COPY_POOLS ? num_pools - first : COPY_POOLS;
        for (int i = 0; i < p.num_pools; ++i) p.pools[i] = static_cast<uint4*>(pools[first + i]);
        const long long items = p.pieces * p.num_pools * F, most = 152ll * 8;
        const kda_status st = launch_early(page_copy_kernel, dim3((unsigned)(items < most ? items : most)), COPY_THREADS, 0, stream, p);
        if (st != KDA_OK) return st;
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
    const long long cells = (long long)N * table_width;   // at most, as the lengths are on the device
    if (cells <= FREE_ALONE) return launch_early(page_free_kernel<true>, dim3(PG_CTAS), PG_THREADS, 0, stream, p);
    const long long blocks = ((long long)num_pages / 4 + 255) / 256 + 1;
    kda_status st = launch_early(page_owners_kernel, dim3((unsigned)(blocks < 152 * 8 ? blocks : 152 * 8)), 256, 0, stream, p);
    if (st != KDA_OK) return st;
    const int warps = 152 * 8 * 4, fit = PG_MOST / table_width;   // (a warp counts its rows' cells in 32 bits)
    int rows = N <= warps ? 1 : N / warps < 32 ? N / warps : 32;
    rows = rows < fit ? rows : fit;
    const long long groups = ((long long)N + 8ll * rows - 1) / (8ll * rows);
    st = launch_early(page_release_kernel, dim3((unsigned)(groups < 152 * 8 ? groups : 152 * 8)), 256, 0, stream, p, rows);
    if (st != KDA_OK) return st;
    return launch_early(page_free_kernel<false>, dim3(PG_CTAS), PG_THREADS, 0, stream, p);
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
    if (p.status && !succeeded(cudaMemsetAsync(p.status, 0, WS_CLEAR, stream))) return KDA_ERR_CUDA;
    const long long cells = (long long)N * table_width;
    if (num_pages <= CP_MOST) {
        const int groups = (num_pages + CP_GROUP - 1) / CP_GROUP, bytes = groups * CP_GROUP_BYTES;
        // (the limit is the kernel's, for all threads that call it: the same for every pool)
        if (!succeeded(cudaFuncSetAttribute(page_compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, CP_MOST / CP_GROUP * CP_GROUP_BYTES)))
            return KDA_ERR_CUDA;
        // an item a thread, though each CTA reads the whole free list (8192 pages, 256 rows of 32: 6 us, with four 11)
        const long long items = cells > num_pages ? cells : num_pages, ctas = (items + PG_THREADS - 1) / PG_THREADS;
        return launch_early(page_compact_kernel, dim3((unsigned)(ctas < 152 ? ctas : 152)), PG_THREADS, bytes, stream, p, table_out);
    }
    const kda_status st = launch(page_compact_large_kernel, dim3(PG_CTAS), PG_THREADS, stream, p);
    const long long blocks = (cells + 255) / 256, most = 152ll * 8;
    if (st != KDA_OK || blocks == 0) return st;
    return launch(page_remap_kernel, dim3((unsigned)(blocks < most ? blocks : most)), 256, stream, p, table_out);
}

}  // extern "C"
