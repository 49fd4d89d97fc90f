// The paged latent cache's bookkeeping: new rows into their slots
// (kda_latent_append) and the block tables and slot map of a step
// (kda_block_tables), with their C entry points.
#include <cstdint>

#include "kda.h"
#include "kda_latent.cuh"

namespace kda {

namespace {

// One warp per row: 72 pieces of 16 bytes, two of the latent channels' 64 a
// lane and one of the positional channels' 8 for lanes 0-7.
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

constexpr int TAB_THREADS = 1024;

// Inclusive prefix sum over the CTA.
__device__ long long cta_scan(long long x, long long* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    long long before = 0;
    for (int w = 0; w < warp; ++w) before += warp_sums[w];
    return x + before;
}

__global__ void block_tables_kernel(TableParams p) {
    __shared__ long long sums[32];
    __shared__ int2 seq_at[TAB_THREADS];       // (first token, first free entry) of the chunk's sequences
    __shared__ int2 seq_len[TAB_THREADS];      // (cached rows, new rows)
    long long tok0 = 0, page0 = 0;
    const long long head = p.free_head[0];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ps = p.page_size;
    bool bad = false;
    for (int base = 0; base < p.N; base += TAB_THREADS) {
        const int n = base + threadIdx.x;
        int a = 0, b = 0;
        long long take = 0;
        if (n < p.N) {
            a = p.lens[n];
            b = p.fresh[n];
            if (a < 0 || b < 0 || (long long)a + b > INT32_MAX) {
                bad = true;
                a = a < 0 ? 0 : a;
                b = b < 0 || (long long)a + b > INT32_MAX ? 0 : b;
            }
            const long long held = ((long long)a + ps - 1) / ps, want = ((long long)a + b + ps - 1) / ps;
            bad |= want > p.width;
            take = max(0ll, min(want, (long long)p.width) - held);
        }
        const long long tok = cta_scan(b, sums), pg = cta_scan(take, sums);
        seq_at[threadIdx.x] = make_int2((int)min(tok0 + tok - b, (long long)INT32_MAX), (int)min(page0 + pg - take, (long long)INT32_MAX));
        seq_len[threadIdx.x] = make_int2(a, b);
        if (n < p.N) {
            p.cu[n] = seq_at[threadIdx.x].x;
            p.lens_out[n] = a + b;
        }
        __syncthreads();
        for (int i = warp; i < min(TAB_THREADS, p.N - base); i += TAB_THREADS / 32) {
            const int la = seq_len[i].x, lb = seq_len[i].y;
            const int held = (int)(((long long)la + ps - 1) / ps);
            int32_t* row = p.table + (long long)(base + i) * p.width;
            const int want = (int)min(((long long)la + lb + ps - 1) / ps, (long long)p.width);
            for (int c = held + lane; c < want; c += 32) {
                const long long at = head + seq_at[i].y + c - held;
                const bool ok = at >= 0 && at < p.num_free;
                bad |= !ok;
                row[c] = ok ? p.free_pages[at] : -1;
            }
            for (int k = lane; k < lb; k += 32) {
                const long long t = (long long)seq_at[i].x + k;
                if (t >= p.num_tokens) {
                    bad = true;
                    break;
                }
                const int pos = la + k, c = pos / ps;
                int page = -1;
                if (c < held) page = c < p.width ? row[c] : -1;
                else if (c < p.width) {
                    const long long at = head + seq_at[i].y + c - held;
                    if (at >= 0 && at < p.num_free) page = p.free_pages[at];
                }
                bad |= page < 0;
                p.slots[t] = page < 0 ? -1 : (int64_t)page * ps + pos % ps;
            }
        }
        __syncthreads();
        if (threadIdx.x == TAB_THREADS - 1) sums[0] = tok, sums[1] = pg;
        __syncthreads();
        tok0 += sums[0];
        page0 += sums[1];
        __syncthreads();
    }
    for (long long t = tok0 + threadIdx.x; t < p.num_tokens; t += TAB_THREADS) p.slots[t] = -1;
    if (threadIdx.x == 0) {
        p.cu[p.N] = (int)min(tok0, (long long)INT32_MAX);
        p.head_out[0] = (int)max(min(head + page0, (long long)p.num_free), min(head, (long long)p.num_free));
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
    block_tables_kernel<<<1, TAB_THREADS, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
