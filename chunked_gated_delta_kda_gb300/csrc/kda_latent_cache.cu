// The paged latent cache's bookkeeping: new rows into their slots
// (kda_latent_append) and the block tables and slot map of a step
// (kda_block_tables), with their C entry points.
#include <cstdint>

#include "kda.h"
#include "kda_latent.cuh"

namespace kda {

namespace {

// One warp per row: 72 pieces of 16 bytes, two of the latent channels' 64 a
// lane and one of the positional channels' 8 for lanes 0-7.  256 rows 2.1 us (a
// launch), 9192 rows 4.1 us (5.1 TB/s), 65536 rows 27 us (5.5 TB/s).
template <typename T>
__global__ void latent_append_kernel(const T* rows, long long stride, const int64_t* slots, const T* weight, float eps,
                                     T* cache, long long num_slots, int count, uint32_t* status) {
    const int lane = threadIdx.x & 31;
    const long long t = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (t >= count) return;
    const long long slot = slots[t];
    if (slot < 0) return;
    if (slot >= num_slots) {
        if (lane == 0) set_status(status, STATUS_BAD_PAGE);
        return;
    }
    const T* src = rows + t * stride;
    T* dst = cache + slot * LAT_ROW;
    uint4 piece[2], pe;
    piece[0] = reinterpret_cast<const uint4*>(src)[lane];
    piece[1] = reinterpret_cast<const uint4*>(src)[lane + 32];
    if (lane < 8) pe = reinterpret_cast<const uint4*>(src)[64 + lane];
    if (weight != nullptr) {
        float x[16], sq = 0.f;
        const T* e = reinterpret_cast<const T*>(piece);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = to_f(e[i]);
            sq += x[i] * x[i];
        }
        const float r = rsqrtf(warp_sum(sq) * (1.f / LAT_C) + eps);
        uint4 wp[2] = {reinterpret_cast<const uint4*>(weight)[lane], reinterpret_cast<const uint4*>(weight)[lane + 32]};
        const T* w = reinterpret_cast<const T*>(wp);
        T* out = reinterpret_cast<T*>(piece);
#pragma unroll
        for (int i = 0; i < 16; ++i) out[i] = from_f<T>(x[i] * r * to_f(w[i]));
    }
    reinterpret_cast<uint4*>(dst)[lane] = piece[0];
    reinterpret_cast<uint4*>(dst)[lane + 32] = piece[1];
    if (lane < 8) reinterpret_cast<uint4*>(dst)[64 + lane] = pe;
}

struct TableParams {
    const int32_t* lens;
    const int32_t* fresh;
    int32_t* table;
    const int32_t* free_pages;
    const int32_t* free_head;
    int64_t* slots;
    int32_t* cu;
    int32_t* lens_out;
    int32_t* head_out;
    uint32_t* status;
    int width, num_free, page_size, num_tokens, N;
};

// Tables of one step.  Every CTA takes the prefix sums of all sequences'
// tokens and pages itself (a few microseconds of latency, in place of a second
// launch), a chunk of sequences at a time; then the tokens, and the pages, are
// spread over all threads of the grid, each finding its sequence by bisection
// in shared memory.  So one long prompt is written as fast as many short ones.
// A page taken in this step is read from the free list, not from the table
// cell that another thread writes.  Bound by latency: 256 sequences with a
// token each 4.6 us, 2048 with 525 thousand tokens (4.5 MB) 10.9 us; 296 us by
// one CTA, a warp a sequence.
constexpr int TAB_THREADS = 512;
constexpr int TAB_SEQS = 2048;                  // sequences of a chunk
constexpr int TAB_PER = TAB_SEQS / TAB_THREADS;

// The last i in [0, n) with a[i] <= x (a[0] <= x).
__device__ __forceinline__ int last_not_above(const long long* a, int n, long long x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(TAB_THREADS) block_tables_kernel(const __grid_constant__ TableParams p) {
    __shared__ long long tok_at[TAB_SEQS + 1], page_at[TAB_SEQS + 1];   // first token and page of each sequence
    __shared__ int lens[TAB_SEQS];
    __shared__ long long sums[2][TAB_THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ps = p.page_size;
    const int shift = 31 - __clz(ps);
    const long long head = p.free_head[0], stride = (long long)gridDim.x * TAB_THREADS;
    const long long me = (long long)blockIdx.x * TAB_THREADS + tid;
    long long tok0 = 0, page0 = 0;              // of the chunk
    bool bad = false;
    auto held_of = [&](int len) { return (int)(((long long)len + ps - 1) >> shift); };
    auto free_page = [&](long long at) {
        at += head;
        const bool ok = at >= 0 && at < p.num_free;
        return ok ? p.free_pages[at] : -1;
    };
    for (int base = 0; base < p.N; base += TAB_SEQS) {
        const int count = min(TAB_SEQS, p.N - base);
        int a[TAB_PER], b[TAB_PER];
        long long take[TAB_PER], toks = 0, pages = 0;
#pragma unroll
        for (int k = 0; k < TAB_PER; ++k) {
            const int i = TAB_PER * tid + k;
            a[k] = i < count ? p.lens[base + i] : 0;
            b[k] = i < count ? p.fresh[base + i] : 0;
            if (a[k] < 0 || b[k] < 0 || (long long)a[k] + b[k] > INT32_MAX) {
                bad = true;
                a[k] = max(a[k], 0);
                if (b[k] < 0 || (long long)a[k] + b[k] > INT32_MAX) b[k] = 0;
            }
            const int want = held_of(a[k] + (long long)b[k] > INT32_MAX ? a[k] : a[k] + b[k]);
            bad |= want > p.width;
            take[k] = max(0, min(want, p.width) - held_of(a[k]));
            toks += b[k];
            pages += take[k];
        }
        long long x = toks, y = pages;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, x, d), v = __shfl_up_sync(0xffffffffu, y, d);
            if (lane >= d) x += u, y += v;
        }
        __syncthreads();                        // the chunk before is done with shared memory
        if (lane == 31) sums[0][warp] = x, sums[1][warp] = y;
        __syncthreads();
        x += tok0 - toks;
        y += page0 - pages;
        for (int w = 0; w < warp; ++w) x += sums[0][w], y += sums[1][w];
#pragma unroll
        for (int k = 0; k < TAB_PER; ++k) {
            const int i = TAB_PER * tid + k;
            tok_at[i] = x;
            page_at[i] = y;
            lens[i] = a[k];
            if (blockIdx.x == 0 && i < count) {
                p.cu[base + i] = (int)min(x, (long long)INT32_MAX);
                p.lens_out[base + i] = a[k] + b[k];
            }
            x += b[k];
            y += take[k];
        }
        if (tid == TAB_THREADS - 1) tok_at[TAB_SEQS] = x, page_at[TAB_SEQS] = y;
        __syncthreads();
        const long long tok1 = tok_at[TAB_SEQS], page1 = page_at[TAB_SEQS];
        for (long long q = page0 + me; q < page1; q += stride) {
            const int i = last_not_above(page_at, count, q);
            const int page = free_page(q);
            bad |= page < 0;
            p.table[(long long)(base + i) * p.width + held_of(lens[i]) + (q - page_at[i])] = page;
        }
        for (long long t = tok0 + me; t < min(tok1, (long long)p.num_tokens); t += stride) {
            const int i = last_not_above(tok_at, count, t);
            const int pos = lens[i] + (int)(t - tok_at[i]), cell = pos >> shift, held = held_of(lens[i]);
            int page = -1;
            if (cell < p.width)
                page = cell < held ? p.table[(long long)(base + i) * p.width + cell] : free_page(page_at[i] + cell - held);
            bad |= page < 0;
            p.slots[t] = page < 0 ? -1 : ((int64_t)page << shift) + (pos & (ps - 1));
        }
        tok0 = tok1;
        page0 = page1;
    }
    for (long long t = tok0 + me; t < p.num_tokens; t += stride) p.slots[t] = -1;
    if (me == 0) {
        bad |= tok0 > p.num_tokens;
        p.cu[p.N] = (int)min(tok0, (long long)INT32_MAX);
        p.head_out[0] = (int)min(head + page0, (long long)p.num_free);
    }
    if (bad) set_status(p.status, STATUS_BAD_PAGE);
}

bool off(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

}  // namespace

}  // namespace kda

extern "C" {

kda_status kda_latent_append(const void* rows, long long row_stride, const int64_t* slots, const void* norm_weight,
                             float eps, void* cache, long long num_slots, int T, unsigned flags, void* workspace,
                             cudaStream_t stream) {
    using namespace kda;
    if (T < 0 || num_slots < 0 || (flags & ~KDA_FLAG_FP16) != 0u || off(workspace, 256)) return KDA_ERR_INVALID_ARG;
    if (T > 0 && (!rows || !slots || !cache)) return KDA_ERR_INVALID_ARG;
    if (row_stride < LAT_ROW || row_stride % 8 != 0) return KDA_ERR_INVALID_ARG;
    if (norm_weight && !(eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    if (off(rows, 16) || off(cache, 16) || off(norm_weight, 16) || off(slots, 8)) return KDA_ERR_INVALID_ARG;
    uint32_t* status = static_cast<uint32_t*>(workspace);
    if (status && cudaMemsetAsync(status, 0, WS_CLEAR, stream) != cudaSuccess) return KDA_ERR_CUDA;
    if (T == 0) return KDA_OK;
    const unsigned grid = (unsigned)((T + 3ll) / 4);
    if (flags & KDA_FLAG_FP16)
        latent_append_kernel<__half><<<grid, 128, 0, stream>>>(
            static_cast<const __half*>(rows), row_stride, slots, static_cast<const __half*>(norm_weight), eps,
            static_cast<__half*>(cache), num_slots, T, status);
    else
        latent_append_kernel<__nv_bfloat16><<<grid, 128, 0, stream>>>(
            static_cast<const __nv_bfloat16*>(rows), row_stride, slots, static_cast<const __nv_bfloat16*>(norm_weight),
            eps, static_cast<__nv_bfloat16*>(cache), num_slots, T, status);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_block_tables(const int32_t* seq_lens, const int32_t* new_lens, int32_t* block_table, int table_width,
                            const int32_t* free_pages, int num_free, const int32_t* free_head, int page_size,
                            int64_t* slot_mapping, int num_tokens, int32_t* cu_seqlens, int32_t* seq_lens_out,
                            int32_t* free_head_out, int N, void* workspace, cudaStream_t stream) {
    using namespace kda;
    if (N < 1 || table_width < 0 || num_free < 0 || num_tokens < 0 || page_size < 1 || (page_size & (page_size - 1)) != 0)
        return KDA_ERR_INVALID_ARG;
    if (!seq_lens || !new_lens || !free_head || !cu_seqlens || !seq_lens_out || !free_head_out ||
        (table_width > 0 && !block_table) || (num_free > 0 && !free_pages) || (num_tokens > 0 && !slot_mapping))
        return KDA_ERR_INVALID_ARG;
    if (off(seq_lens, 4) || off(new_lens, 4) || off(block_table, 4) || off(free_pages, 4) || off(free_head, 4) ||
        off(slot_mapping, 8) || off(cu_seqlens, 4) || off(seq_lens_out, 4) || off(free_head_out, 4) ||
        off(workspace, 256))
        return KDA_ERR_INVALID_ARG;
    uint32_t* status = static_cast<uint32_t*>(workspace);
    if (status && cudaMemsetAsync(status, 0, WS_CLEAR, stream) != cudaSuccess) return KDA_ERR_CUDA;
    TableParams p{seq_lens, new_lens,   block_table,  free_pages,    free_head,   slot_mapping, cu_seqlens,
                  seq_lens_out, free_head_out, status, table_width, num_free, page_size, num_tokens, N};
    // eight tokens a thread before another CTA repeats the prefix sums
    const int grid = (int)(((long long)num_tokens + 8ll * TAB_THREADS - 1) / (8ll * TAB_THREADS));
    block_tables_kernel<<<grid < 1 ? 1 : grid > 152 ? 152 : grid, TAB_THREADS, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
