// C ABI of latent attention (expanded forward and backward, absorbed decode):
// host-side argument checks, workspace sizing and launches.  See
// include/kda.h for the contract.
#include <cmath>
#include <cstdint>

#include "kda.h"
#include "kda_latent_decode.cuh"

namespace kda {
uint32_t debug_wait_limit();
cudaError_t launch_latent_fwd(const LatentParams& p, bool fp16, cudaStream_t stream);
cudaError_t launch_latent_bwd(const LatentParams& p, bool fp16, cudaStream_t stream);
cudaError_t launch_latent_decode(const DecodeParams& p, bool fp16, cudaStream_t stream);
unsigned long long latent_decode_scratch(int N, int S, int H);
unsigned long long latent_share_bytes(int B, int Tq, int Tk, int H, int N);
unsigned long long latent_aux_floats(int B, int Tq, int H, int N);
}  // namespace kda

namespace {

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }
bool off256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) != 0; }

unsigned long long round256(unsigned long long b) { return (b + 255ull) / 256ull * 256ull; }

float scale_of(float s) { return s > 0.f && !std::isnan(s) ? s : 1.0f / std::sqrt((float)kda::LAT_QK); }

// (the last line: a CTA a tile slot and head, in one dimension of a grid)
bool sizes_ok(int B, int Tq, int Tk, int H, int N) {
    return B >= 1 && Tq >= 0 && Tk >= 0 && H >= 1 && N >= 1 && H <= 65535 && N <= 65535 &&
           (long long)B * Tq < (1ll << 31) && (long long)B * Tk < (1ll << 31) &&
           ((long long)B * (Tq > Tk ? Tq : Tk) / kda::LAT_TILE + N) * H < (1ll << 31);
}

// The checks that forward and backward share.
kda_status check_common(const void* q, const void* kv, const void* k_pe, long long k_pe_stride, const int32_t* cu_q,
                        const int32_t* cu_k, int B, int Tq, int Tk, int H, int N, unsigned flags, const void* ws) {
    if (!sizes_ok(B, Tq, Tk, H, N) || (flags & ~(KDA_FLAG_FP16 | KDA_FLAG_CAUSAL)) != 0u) return KDA_ERR_INVALID_ARG;
    if ((cu_q == nullptr) != (cu_k == nullptr)) return KDA_ERR_INVALID_ARG;
    if (cu_q == nullptr ? N != B : B != 1) return KDA_ERR_INVALID_ARG;
    if ((Tq > 0 && !q) || (Tk > 0 && (!kv || !k_pe))) return KDA_ERR_INVALID_ARG;
    if (k_pe_stride < kda::LAT_P || k_pe_stride % 8 != 0 || k_pe_stride >= (1ll << 38)) return KDA_ERR_INVALID_ARG;
    if (off16(q) || off16(kv) || off16(k_pe) || off4(cu_q) || off4(cu_k) || off256(ws)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_latent_fwd_workspace_bytes(int B, int Tq, int Tk, int H, int N) {
    return sizes_ok(B, Tq, Tk, H, N) ? (size_t)(kda::WS_HEADER + kda::latent_share_bytes(B, Tq, Tk, H, N)) : 0;
}

kda_status kda_latent_fwd(const void* q, const void* kv, const void* k_pe, long long k_pe_stride, float scale,
                          const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, void* o, float* lse, int B,
                          int Tq, int Tk, int H, int N, unsigned flags, void* workspace, cudaStream_t stream) {
    return kda_latent_fwd_ws(q, kv, k_pe, k_pe_stride, scale, cu_seqlens_q, cu_seqlens_k, o, lse, B, Tq, Tk, H, N, flags,
                             workspace, workspace ? kda::WS_HEADER : 0, stream);
}

kda_status kda_latent_fwd_ws(const void* q, const void* kv, const void* k_pe, long long k_pe_stride, float scale,
                             const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, void* o, float* lse, int B,
                             int Tq, int Tk, int H, int N, unsigned flags, void* workspace, size_t workspace_bytes,
                             cudaStream_t stream) {
    const kda_status st = check_common(q, kv, k_pe, k_pe_stride, cu_seqlens_q, cu_seqlens_k, B, Tq, Tk, H, N, flags,
                                       workspace);
    if (st != KDA_OK) return st;
    if ((Tq > 0 && !o) || off16(o) || off4(lse)) return KDA_ERR_INVALID_ARG;
    if (workspace && workspace_bytes < kda::WS_HEADER) return KDA_ERR_INVALID_ARG;
    kda::LatentParams p{};
    const unsigned long long share = workspace && cu_seqlens_q ? kda::latent_share_bytes(B, Tq, Tk, H, N) : 0;
    if (share > 0 && workspace_bytes >= kda::WS_HEADER + share) {
        uint8_t* at = static_cast<uint8_t*>(workspace) + kda::WS_HEADER;
        p.share_items = reinterpret_cast<int4*>(at);
        p.share_parts = reinterpret_cast<float*>(at + kda::LATENT_SHARE_ITEMS * 16ull);
    }
    p.q = q;
    p.kv = kv;
    p.k_pe = k_pe;
    p.k_pe_stride = k_pe_stride;
    p.o_out = o;
    p.lse_out = lse;
    p.cu_q = cu_seqlens_q;
    p.cu_k = cu_seqlens_k;
    p.status = static_cast<uint32_t*>(workspace);
    p.scale = scale_of(scale);
    p.Tq = Tq;
    p.Tk = Tk;
    p.H = H;
    p.N = N;
    p.causal = (flags & KDA_FLAG_CAUSAL) != 0u;
    p.wait_limit = kda::debug_wait_limit();
    // (with shared key ranges the first kernel clears it)
    if (workspace && (Tq == 0 || !p.share_items) && cudaMemsetAsync(workspace, 0, kda::WS_CLEAR, stream) != cudaSuccess)
        return KDA_ERR_CUDA;
    if (Tq == 0) return KDA_OK;
    return kda::launch_latent_fwd(p, (flags & KDA_FLAG_FP16) != 0u, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

// Header, the queries' tables (latent_aux_kernel), the per-head gradients of k_pe.
size_t kda_latent_bwd_workspace_bytes(int B, int Tq, int Tk, int H, int N) {
    if (!sizes_ok(B, Tq, Tk, H, N)) return 0;
    return (size_t)(kda::WS_HEADER + round256(kda::latent_aux_floats(B, Tq, H, N) * 4ull) +
                    (unsigned long long)B * Tk * H * kda::LAT_P * 4ull);
}

kda_status kda_latent_bwd(const void* q, const void* kv, const void* k_pe, long long k_pe_stride, const void* o,
                          const float* lse, const void* dout, float scale, const int32_t* cu_seqlens_q,
                          const int32_t* cu_seqlens_k, void* dq, void* dkv, void* dk_pe, int B, int Tq, int Tk,
                          int H, int N, unsigned flags, void* workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
    const kda_status st = check_common(q, kv, k_pe, k_pe_stride, cu_seqlens_q, cu_seqlens_k, B, Tq, Tk, H, N, flags,
                                       workspace);
    if (st != KDA_OK) return st;
    if (!workspace || workspace_bytes < kda_latent_bwd_workspace_bytes(B, Tq, Tk, H, N)) return KDA_ERR_INVALID_ARG;
    if ((Tq > 0 && (!o || !lse || !dout || !dq)) || (Tk > 0 && (!dkv || !dk_pe))) return KDA_ERR_INVALID_ARG;
    if (off16(o) || off4(lse) || off16(dout) || off16(dq) || off16(dkv) || off16(dk_pe)) return KDA_ERR_INVALID_ARG;
    kda::LatentParams p{};
    p.q = q;
    p.kv = kv;
    p.k_pe = k_pe;
    p.k_pe_stride = k_pe_stride;
    p.o = o;
    p.lse = lse;
    p.dout = dout;
    p.dq = dq;
    p.dkv = dkv;
    p.dk_pe = dk_pe;
    p.cu_q = cu_seqlens_q;
    p.cu_k = cu_seqlens_k;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.status = reinterpret_cast<uint32_t*>(ws);
    p.aux = reinterpret_cast<float*>(ws + kda::WS_HEADER);
    p.dpe_part = reinterpret_cast<float*>(ws + kda::WS_HEADER + round256(kda::latent_aux_floats(B, Tq, H, N) * 4ull));
    p.scale = scale_of(scale);
    p.Tq = Tq;
    p.Tk = Tk;
    p.H = H;
    p.N = N;
    p.causal = (flags & KDA_FLAG_CAUSAL) != 0u;
    p.wait_limit = kda::debug_wait_limit();
    if (cudaMemsetAsync(workspace, 0, kda::WS_CLEAR, stream) != cudaSuccess) return KDA_ERR_CUDA;
    return kda::launch_latent_bwd(p, (flags & KDA_FLAG_FP16) != 0u, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

static bool decode_sizes_ok(int N, int S, int H) {
    return N >= 1 && S >= 1 && H >= 1 && N <= 65535 && S <= 65535 && H <= 65535 && (long long)N * S * H < (1ll << 31);
}

size_t kda_latent_decode_workspace_bytes(int N, int S, int H) {
    return decode_sizes_ok(N, S, H) ? (size_t)kda::latent_decode_scratch(N, S, H) : 0;
}

kda_status kda_latent_decode(const void* q, const void* cache, int num_pages, int page_size,
                             const int32_t* block_table, int table_width, const int32_t* seq_lens, float scale,
                             void* o, float* lse, int N, int S, int H, unsigned flags, void* workspace,
                             size_t workspace_bytes, cudaStream_t stream) {
    if (!decode_sizes_ok(N, S, H) || (flags & ~KDA_FLAG_FP16) != 0u) return KDA_ERR_INVALID_ARG;
    if (num_pages < 1 || table_width < 1) return KDA_ERR_INVALID_ARG;
    if (page_size != 16 && page_size != 32 && (page_size < 64 || page_size % 64 != 0)) return KDA_ERR_INVALID_ARG;
    if ((long long)num_pages * page_size >= (1ll << 31) || (long long)table_width * page_size >= (1ll << 31))
        return KDA_ERR_INVALID_ARG;
    if (!q || !cache || !block_table || !seq_lens || !o || !workspace) return KDA_ERR_INVALID_ARG;
    if (off16(q) || off16(cache) || off4(block_table) || off4(seq_lens) || off16(o) || off4(lse) || off256(workspace))
        return KDA_ERR_INVALID_ARG;
    if (workspace_bytes < kda_latent_decode_workspace_bytes(N, S, H)) return KDA_ERR_INVALID_ARG;
    kda::DecodeParams p{};
    p.q = q;
    p.cache = cache;
    p.table = block_table;
    p.lens = seq_lens;
    p.o = o;
    p.lse = lse;
    p.workspace = static_cast<uint8_t*>(workspace);
    p.status = static_cast<uint32_t*>(workspace);
    p.scale = scale_of(scale);
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.table_width = table_width;
    p.N = N;
    p.S = S;
    p.H = H;
    p.wait_limit = kda::debug_wait_limit();
    return kda::launch_latent_decode(p, (flags & KDA_FLAG_FP16) != 0u, stream) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
