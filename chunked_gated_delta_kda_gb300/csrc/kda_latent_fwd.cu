// Expanded latent attention, forward: one warp per (query, head), the keys in
// order, with the running maximum and sum of the softmax.
#include "kda_latent.cuh"

namespace kda {

namespace {

template <typename T>
__global__ void latent_fwd_kernel(LatentParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int n, j;
    latent_slot(p.cu_q, p.Tq, p.N, blockIdx.x, n, j);
    LatentSeq s;
    if (!latent_seq(p, n, s)) return;
    const int h = blockIdx.y;
    for (int r = warp; r < LAT_TILE; r += blockDim.x >> 5) {
        const int i = j * LAT_TILE + r;
        if (i >= s.lq) return;
        const T* q = static_cast<const T*>(p.q) + ((s.q0 + i) * p.H + h) * LAT_QK;
        float qv[6], acc[4] = {0.f, 0.f, 0.f, 0.f};
        for (int e = 0; e < 6; ++e) qv[e] = to_f(q[lane + 32 * e]) * p.scale;
        const int last = p.causal ? min(s.lk, i + s.lk - s.lq + 1) : s.lk;
        float m = -INFINITY, l = 0.f;
        for (int k = 0; k < last; ++k) {
            const T* kv = static_cast<const T*>(p.kv) + ((s.k0 + k) * p.H + h) * LAT_KV;
            const T* pe = static_cast<const T*>(p.k_pe) + (s.k0 + k) * p.k_pe_stride;
            float x = 0.f;
            for (int e = 0; e < 4; ++e) x += qv[e] * to_f(kv[lane + 32 * e]);
            for (int e = 0; e < 2; ++e) x += qv[4 + e] * to_f(pe[lane + 32 * e]);
            x = warp_sum(x);
            const float mn = fmaxf(m, x), c = mn == -INFINITY ? 1.f : expf(m - mn), w = mn == -INFINITY ? 0.f : expf(x - mn);
            l = l * c + w;
            for (int e = 0; e < 4; ++e) acc[e] = acc[e] * c + w * to_f(kv[LAT_N + lane + 32 * e]);
            m = mn;
        }
        T* o = static_cast<T*>(p.o_out) + ((s.q0 + i) * p.H + h) * LAT_V;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        for (int e = 0; e < 4; ++e) o[lane + 32 * e] = from_f<T>(l > 0.f ? acc[e] * inv : 0.f);
        if (lane == 0 && p.lse_out) p.lse_out[(s.q0 + i) * p.H + h] = l > 0.f ? m + logf(l) : -INFINITY;
    }
}

}  // namespace

cudaError_t launch_latent_fwd(const LatentParams& p, bool fp16, cudaStream_t stream) {
    const int slots = latent_slots(p.cu_q != nullptr, p.Tq, p.N);
    const dim3 grid(slots, p.H);
    if (fp16) latent_fwd_kernel<__half><<<grid, 256, 0, stream>>>(p);
    else latent_fwd_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace kda
