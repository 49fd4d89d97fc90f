// Pages that several requests own: forking, freeing, compacting and copying
// (kda_page_fork, kda_page_free, kda_page_compact, kda_page_copy), with their
// C entry points.  See include/kda.h for the contract.
//
// The first three are bookkeeping of a few thousand words whose steps depend
// on each other (owners counted before pages are given back, pages numbered
// before tables are rewritten).  Each runs as one cluster of eight CTAs with
// cluster barriers between the steps: one launch.  What one CTA writes and
// another reads goes through the L2 (atomics, __stcg, __ldcg).
#include <cstdint>

#include "kda.h"
#include "kda_latent_mma.cuh"

namespace kda {

namespace {

constexpr int PG_CTAS = 8;
constexpr int PG_THREADS = 512;
constexpr int PG_ALL = PG_CTAS * PG_THREADS;
constexpr int PG_PER = 8;                        // pages of a thread, in a row
constexpr int PG_CHUNK = PG_THREADS * PG_PER;

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
    int32_t* scratch;
    uint32_t* status;
    int width, num_pages, num_free, page_size, N, F;
};

// A row's pages, its length clipped to the table's columns.
__device__ __forceinline__ int row_pages(const PageParams& p, int len, bool& bad) {
    const long long most = (long long)p.width * p.page_size;
    bad |= len < 0 || len > most;
    return (int)((max(0ll, min((long long)len, most)) + p.page_size - 1) / p.page_size);
}

__device__ __forceinline__ void copy_words(const int32_t* from, int32_t* to, int count, int me) {
    if (((reinterpret_cast<uintptr_t>(from) | reinterpret_cast<uintptr_t>(to)) & 15u) == 0) {
        const int quads = count >> 2;
#pragma unroll 4
        for (int i = me; i < quads; i += PG_ALL) __stcg(reinterpret_cast<int4*>(to) + i, __ldg(reinterpret_cast<const int4*>(from) + i));
        if (me < (count & 3)) __stcg(to + 4 * quads + me, __ldg(from + 4 * quads + me));
        return;
    }
#pragma unroll 4
    for (int i = me; i < count; i += PG_ALL) __stcg(to + i, __ldg(from + i));
}

__device__ __forceinline__ void fill_words(int32_t* to, int value, int count, int me) {
    for (int i = me; i < count; i += PG_ALL) __stcg(to + i, value);
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
    int before = x - mine;
    total = 0;
#pragma unroll
    for (int w = 0; w < PG_THREADS / 32; ++w) {
        const int s = sums[w];
        if (w < warp) before += s;
        total += s;
    }
    return before;
}

// `mine` of every CTA of the cluster (thread 0's): the sum of those of lower
// rank, and of all.  Ends in a cluster barrier.
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
__global__ void __cluster_dims__(PG_CTAS, 1, 1) __launch_bounds__(PG_THREADS) page_fork_kernel(const __grid_constant__ PageParams p) {
    __shared__ int sums[PG_THREADS / 32];
    __shared__ int4 entries[PG_THREADS];         // parent (-1: skipped), child, tokens, place among the own pages (-1: none)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)cluster_rank(), me = rank * PG_THREADS + tid;
    const int head = p.free_head[0];
    bool bad = false;
    if (me == 0 && p.status) __stcg(p.status, 0u);
    copy_words(p.refs, p.refs_out, p.num_pages, me);
    copy_words(p.lens, p.lens_out, p.N, me);
    fill_words(p.scratch, INT32_MAX, p.N, me);
    cluster_barrier();
    // each child's first entry
    auto in_range = [&](int a, int c) { return a >= 0 && a < p.N && c < p.N; };
    for (int i = me; i < p.F; i += PG_ALL) {
        const int c = p.children[i];
        if (c >= 0 && in_range(p.parents[i], c)) atomicMin(p.scratch + c, i);
    }
    cluster_barrier();
    int taken = 0;
    for (int base = 0; base < p.F; base += PG_THREADS) {
        const int i = base + tid;
        int4 e = make_int4(-1, -1, 0, -1);
        if (i < p.F) {
            const int a = p.parents[i], c = p.children[i];
            if (c >= 0) {
                if (in_range(a, c) && p.lens[c] == 0 && __ldcg(p.scratch + c) == i) {
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
        __syncthreads();
        for (int k = rank * (PG_THREADS / 32) + warp; k < min(PG_THREADS, p.F - base); k += PG_ALL / 32) {
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
        __syncthreads();
    }
    if (me == 0) p.head_out[0] = (int)max((long long)min(head, 0), min((long long)head + taken, (long long)max(head, p.num_free)));
    if (bad) set_status(p.status, STATUS_BAD_PAGE);
}

// ---- free ----
// The pages of a CTA, PG_CHUNK at a time, in the order of their numbers:
// f(first page of the thread, mask of its pages, how many of the CTA's pages
// before it are in a mask).
template <typename MASK, typename FUNC>
__device__ __forceinline__ int walk_pages(int first, int last, int* sums, MASK mask_of, FUNC f) {
    int running = 0;
    for (int base = first; base < last; base += PG_CHUNK) {
        const int at = base + (int)threadIdx.x * PG_PER;
        const uint32_t mask = at < last ? mask_of(at, min(PG_PER, last - at)) : 0u;
        int total;
        const int before = block_before(__popc(mask), total, sums);
        if (at < last) f(at, min(PG_PER, last - at), mask, running + before);
        running += total;
    }
    return running;
}

// The CTA's pages, in whole eights.
__device__ __forceinline__ void page_range(int num_pages, int& first, int& last) {
    const int each = (int)((((long long)num_pages + PG_CTAS - 1) / PG_CTAS + PG_PER - 1) / PG_PER * PG_PER);
    first = (int)min((long long)num_pages, (long long)cluster_rank() * each);
    last = (int)min((long long)num_pages, (long long)first + each);
}

// PG_PER words from a 16-byte aligned array of the workspace (padded to whole eights).
__device__ __forceinline__ void load_words(const int32_t* from, int (&x)[PG_PER]) {
    const int4 a = __ldcg(reinterpret_cast<const int4*>(from)), b = __ldcg(reinterpret_cast<const int4*>(from) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

__global__ void __cluster_dims__(PG_CTAS, 1, 1) __launch_bounds__(PG_THREADS) page_free_kernel(const __grid_constant__ PageParams p) {
    __shared__ int sums[PG_THREADS / 32], slots[PG_CTAS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)cluster_rank(), me = rank * PG_THREADS + tid;
    const long long head = p.free_head[0];
    bool bad = false;
    if (me == 0 && p.status) __stcg(p.status, 0u);
    fill_words(p.scratch, 0, p.num_pages, me);
    cluster_barrier();
    for (int n = rank * (PG_THREADS / 32) + warp; n < p.N; n += PG_ALL / 32) {
        const int len = p.lens[n], keep = p.keep[n], kept = max(0, min(keep, len));
        bad |= keep != kept;
        const int from = row_pages(p, kept, bad), to = row_pages(p, len, bad);
        if (lane == 0) p.lens_out[n] = kept;
#pragma unroll 4
        for (int col = from + lane; col < to; col += 32) {
            const int page = p.table[(long long)n * p.width + col];
            if (page >= 0 && page < p.num_pages) atomicAdd(p.scratch + page, 1);
            else bad = true;
        }
    }
    cluster_barrier();
    int first, last;
    page_range(p.num_pages, first, last);
    auto freed = [&](int at, int n) {            // the pages that lose their last owner
        int lost[PG_PER];
        load_words(p.scratch + at, lost);
        uint32_t mask = 0;
#pragma unroll
        for (int k = 0; k < PG_PER; ++k)
            if (k < n && lost[k] > 0 && lost[k] > __ldg(p.refs + at + k)) mask |= 1u << k;
        return mask;
    };
    const int mine = walk_pages(first, last, sums, freed, [&](int at, int n, uint32_t mask, int) {
        int lost[PG_PER];
        load_words(p.scratch + at, lost);
#pragma unroll
        for (int k = 0; k < PG_PER; ++k)
            if (k < n) {
                const int had = __ldg(p.refs + at + k);
                bad |= (long long)lost[k] > (long long)max(had, 0) + 1;
                p.refs_out[at + k] = max(had - lost[k], 0);
            }
    });
    int all;
    const int before = cluster_before(mine, all, slots);
    walk_pages(first, last, sums, freed, [&](int at, int, uint32_t mask, int place) {
        long long to = head - all + before + place;
        for (; mask != 0u; mask &= mask - 1, ++to) {
            if (to >= 0 && to < p.num_free) p.free_io[to] = at + __ffs(mask) - 1;
            else bad = true;
        }
    });
    if (me == 0) p.head_out[0] = (int)max(0ll, head - all);
    if (bad) set_status(p.status, STATUS_BAD_PAGE);
}

// ---- compact ----
__global__ void __cluster_dims__(PG_CTAS, 1, 1) __launch_bounds__(PG_THREADS) page_compact_kernel(const __grid_constant__ PageParams p) {
    __shared__ int sums[PG_THREADS / 32], slots[3][PG_CTAS];
    const int rank = (int)cluster_rank(), me = rank * PG_THREADS + (int)threadIdx.x;
    const long long head = p.free_head[0];
    bool bad = false;
    if (me == 0 && p.status) __stcg(p.status, 0u);
    fill_words(p.scratch, 0, p.num_pages, me);
    fill_words(p.pairs, -1, p.num_pages / 2 * 2, me);
    cluster_barrier();
    for (long long i = max(head, 0ll) + me; i < p.num_free; i += PG_ALL) {
        const int page = p.free_pages[i];
        if (page < 0 || page >= p.num_pages || atomicExch(p.scratch + page, 1) != 0) bad = true;
    }
    cluster_barrier();
    int first, last;
    page_range(p.num_pages, first, last);
    auto free_mask = [&](int at, int n) {
        int x[PG_PER];
        load_words(p.scratch + at, x);
        uint32_t mask = 0;
#pragma unroll
        for (int k = 0; k < PG_PER; ++k)
            if (k < n && x[k] != 0) mask |= 1u << k;
        return mask;
    };
    int all, holes;
    const int before = cluster_before(walk_pages(first, last, sums, free_mask, [](int, int, uint32_t, int) {}), all, slots[0]);
    const int used = p.num_pages - all;
    const int upto = min(max(used, first), last);              // the CTA's pages below `used`
    cluster_before(walk_pages(first, upto, sums, free_mask, [](int, int, uint32_t, int) {}), holes, slots[1]);
    // the k-th free page below `used` takes the k-th used one from there on
    auto place = [&](auto f) {
        walk_pages(first, last, sums, free_mask, [&](int at, int n, uint32_t mask, int ahead) {
            int free_before = before + ahead;
#pragma unroll
            for (int k = 0; k < PG_PER; ++k)
                if (k < n) {
                    const int i = at + k;
                    const bool is_free = (mask >> k) & 1u;
                    f(i, is_free, is_free ? free_before : (i - used) - (free_before - holes));
                    free_before += is_free;
                }
        });
    };
    place([&](int i, bool is_free, int k) {
        if (is_free == (i < used)) __stcg(p.pairs + 2ll * k + (is_free ? 1 : 0), i);
    });
    cluster_barrier();
    place([&](int i, bool is_free, int k) {
        int to = i;
        if (is_free) to = -1;
        else if (i >= used) to = __ldcg(p.pairs + 2ll * k + 1);
        p.moved[i] = to;
        if (to >= 0) p.refs_out[to] = __ldg(p.refs + i);
        if (i >= used) p.refs_out[i] = 0;
    });
    for (int i = me; i < p.num_free; i += PG_ALL) {
        const long long to = used + (i - head);
        const bool fits = to < p.num_pages;
        p.free_out[i] = i < head ? p.free_pages[i] : fits ? (int)to : -1;
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

// ---- copy: pieces of 16 KiB of all pairs and pools, dealt to the CTAs ----
constexpr int COPY_POOLS = 64;                   // of one launch
constexpr int COPY_THREADS = 256;
constexpr int COPY_PIECE = COPY_THREADS * 4;     // 16-byte words

struct CopyParams {
    uint4* pools[COPY_POOLS];
    const int32_t* pairs;
    const int32_t* count;
    uint32_t* status;
    long long words;                             // of a page
    int num_pools, num_pages, F;
};

__global__ void __launch_bounds__(COPY_THREADS) page_copy_kernel(const __grid_constant__ CopyParams p) {
    const int pairs = p.count ? max(0, min(p.F, p.count[0])) : p.F;
    const long long pieces = (p.words + COPY_PIECE - 1) / COPY_PIECE, items = pieces * p.num_pools * pairs;
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        const long long pair = item / (pieces * p.num_pools), rest = item - pair * (pieces * p.num_pools);
        const long long pool = rest / pieces, first = (rest - pool * pieces) * COPY_PIECE;
        const int src = p.pairs[2 * pair], dst = p.pairs[2 * pair + 1];
        if (src < 0 || dst < 0) continue;
        if (src >= p.num_pages || dst >= p.num_pages) {
            if (threadIdx.x == 0) set_status(p.status, STATUS_BAD_PAGE);
            continue;
        }
        const uint4* from = p.pools[pool] + src * p.words;
        uint4* to = p.pools[pool] + dst * p.words;
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const long long at = first + threadIdx.x + COPY_THREADS * k;
            if (at < p.words) x[k] = __ldcs(from + at);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const long long at = first + threadIdx.x + COPY_THREADS * k;
            if (at < p.words) __stcs(to + at, x[k]);
        }
    }
}

bool off(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

template <typename... P>
bool missing(const P*... p) { return ((p == nullptr) || ...); }
template <typename... P>
bool off4(const P*... p) { return (off(p, 4) || ...); }

size_t scratch_bytes(int words) { return words < 1 ? 0 : WS_HEADER + ((size_t)words + 7) / 8 * 32; }

// What the three share: sizes, the table, the free list, the workspace.
bool common_ok(const PageParams& p, const void* table, const void* workspace, size_t bytes, size_t need) {
    if (p.N < 1 || p.width < 0 || p.num_pages < 1 || p.num_free < 0 || p.page_size < 1) return false;
    if ((p.width > 0 && !table) || missing(p.lens, p.refs, p.refs_out, p.free_head) || !workspace || bytes < need) return false;
    return !off4(table, p.lens, p.refs, p.refs_out, p.free_head) && !off(workspace, 256);
}

kda_status launched() { return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace

}  // namespace kda

extern "C" {

size_t kda_page_fork_workspace_bytes(int N) { return kda::scratch_bytes(N); }
size_t kda_page_free_workspace_bytes(int num_pages) { return kda::scratch_bytes(num_pages); }
size_t kda_page_compact_workspace_bytes(int num_pages) { return kda::scratch_bytes(num_pages); }

kda_status kda_page_fork(int32_t* block_table, int table_width, const int32_t* seq_lens, const int32_t* parents,
                         const int32_t* children, const int32_t* refs, int num_pages, const int32_t* free_pages,
                         int num_free, const int32_t* free_head, int page_size, int32_t* seq_lens_out,
                         int32_t* refs_out, int32_t* free_head_out, int32_t* pairs, int N, int F, void* workspace,
                         size_t workspace_bytes, cudaStream_t stream) {
    using namespace kda;
    PageParams p{};
    p.table_io = block_table, p.lens = seq_lens, p.parents = parents, p.children = children, p.refs = refs;
    p.free_pages = free_pages, p.free_head = free_head, p.lens_out = seq_lens_out, p.refs_out = refs_out;
    p.head_out = free_head_out, p.pairs = pairs;
    p.width = table_width, p.num_pages = num_pages, p.num_free = num_free, p.page_size = page_size, p.N = N, p.F = F;
    if (!common_ok(p, block_table, workspace, workspace_bytes, kda_page_fork_workspace_bytes(N)) || F < 0) return KDA_ERR_INVALID_ARG;
    if (missing(seq_lens_out, free_head_out) || (F > 0 && missing(parents, children, pairs)) || (num_free > 0 && !free_pages))
        return KDA_ERR_INVALID_ARG;
    if (off4(parents, children, free_pages, seq_lens_out, free_head_out, pairs)) return KDA_ERR_INVALID_ARG;
    p.status = static_cast<uint32_t*>(workspace);
    p.scratch = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + WS_HEADER);
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
    if (p.status && cudaMemsetAsync(p.status, 0, WS_CLEAR, stream) != cudaSuccess) return KDA_ERR_CUDA;
    if (F == 0) return KDA_OK;
    for (int first = 0; first < num_pools; first += COPY_POOLS) {
        p.num_pools = num_pools - first < COPY_POOLS ? num_pools - first : COPY_POOLS;
        for (int i = 0; i < p.num_pools; ++i) p.pools[i] = static_cast<uint4*>(pools[first + i]);
        const long long items = (p.words + COPY_PIECE - 1) / COPY_PIECE * p.num_pools * F, most = 152ll * 8;
        page_copy_kernel<<<(unsigned)(items < most ? items : most), COPY_THREADS, 0, stream>>>(p);
        if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
    }
    return KDA_OK;
}

kda_status kda_page_free(const int32_t* block_table, int table_width, const int32_t* seq_lens,
                         const int32_t* keep_lens, const int32_t* refs, int num_pages, int32_t* free_pages,
                         int num_free, const int32_t* free_head, int page_size, int32_t* seq_lens_out,
                         int32_t* refs_out, int32_t* free_head_out, int N, void* workspace, size_t workspace_bytes,
                         cudaStream_t stream) {
    using namespace kda;
    PageParams p{};
    p.table = block_table, p.lens = seq_lens, p.keep = keep_lens, p.refs = refs, p.free_io = free_pages;
    p.free_head = free_head, p.lens_out = seq_lens_out, p.refs_out = refs_out, p.head_out = free_head_out;
    p.width = table_width, p.num_pages = num_pages, p.num_free = num_free, p.page_size = page_size, p.N = N;
    if (!common_ok(p, block_table, workspace, workspace_bytes, kda_page_free_workspace_bytes(num_pages))) return KDA_ERR_INVALID_ARG;
    if (missing(keep_lens, seq_lens_out, free_head_out) || (num_free > 0 && !free_pages)) return KDA_ERR_INVALID_ARG;
    if (off4(keep_lens, free_pages, seq_lens_out, free_head_out)) return KDA_ERR_INVALID_ARG;
    p.status = static_cast<uint32_t*>(workspace);
    p.scratch = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + WS_HEADER);
    page_free_kernel<<<PG_CTAS, PG_THREADS, 0, stream>>>(p);
    return launched();
}

kda_status kda_page_compact(const int32_t* block_table, int table_width, const int32_t* seq_lens, const int32_t* refs,
                            int num_pages, const int32_t* free_pages, int num_free, const int32_t* free_head,
                            int page_size, int32_t* table_out, int32_t* refs_out, int32_t* free_out, int32_t* pairs,
                            int32_t* count, int32_t* moved, int N, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
    using namespace kda;
    PageParams p{};
    p.table = block_table, p.lens = seq_lens, p.refs = refs, p.free_pages = free_pages, p.free_head = free_head;
    p.refs_out = refs_out, p.free_out = free_out, p.pairs = pairs, p.count = count, p.moved = moved;
    p.width = table_width, p.num_pages = num_pages, p.num_free = num_free, p.page_size = page_size, p.N = N;
    if (!common_ok(p, block_table, workspace, workspace_bytes, kda_page_compact_workspace_bytes(num_pages)))
        return KDA_ERR_INVALID_ARG;
    if (missing(count, moved) || (num_free > 0 && missing(free_pages, free_out)) || (num_pages > 1 && !pairs) ||
        (table_width > 0 && !table_out))
        return KDA_ERR_INVALID_ARG;
    if (off4(free_pages, free_out, pairs, count, moved, table_out)) return KDA_ERR_INVALID_ARG;
    p.status = static_cast<uint32_t*>(workspace);
    p.scratch = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + WS_HEADER);
    page_compact_kernel<<<PG_CTAS, PG_THREADS, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
    const long long blocks = ((long long)N * table_width + 255) / 256, most = 152ll * 8;
    if (blocks == 0) return KDA_OK;
    page_remap_kernel<<<(unsigned)(blocks < most ? blocks : most), 256, 0, stream>>>(p, table_out);
    return launched();
}

}  // extern "C"
