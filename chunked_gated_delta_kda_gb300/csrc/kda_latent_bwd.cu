// Expanded latent attention, backward.  One warp per (query, head) for dq and
// dout . o, one per (key, head) for dk and dv; the shared positional key's
// per-head gradients go to the workspace and are summed in head order.
#include "kda_latent.cuh"

namespace kda {

namespace {

template <typename T>
__global__ void latent_dq_kernel(LatentParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int n, j;
    latent_slot(p.cu_q, p.Tq, p.N, blockIdx.x, LAT_TILE, n, j);
    LatentSeq s;
    if (!latent_seq(p, n, s)) return;
    const int h = blockIdx.y;
    for (int r = warp; r < LAT_TILE; r += blockDim.x >> 5) {
        const int i = j * LAT_TILE + r;
        if (i >= s.lq) return;
        const long long row = (s.q0 + i) * p.H + h;
        const T* q = static_cast<const T*>(p.q) + row * LAT_QK;
        const T* dob = static_cast<const T*>(p.dout) + row * LAT_V;
        const T* ob = static_cast<const T*>(p.o) + row * LAT_V;
        float qv[6], dv[4], acc[6] = {}, delta = 0.f;
        for (int e = 0; e < 6; ++e) qv[e] = to_f(q[lane + 32 * e]) * p.scale;
        for (int e = 0; e < 4; ++e) {
            dv[e] = to_f(dob[lane + 32 * e]);
            delta += dv[e] * to_f(ob[lane + 32 * e]);
        }
        delta = warp_sum(delta);
        if (lane == 0) p.delta[row] = delta;
        const float lse = p.lse[row];
        const int last = p.causal ? min(s.lk, i + s.lk - s.lq + 1) : s.lk;
        for (int k = 0; k < last; ++k) {
            const T* kv = static_cast<const T*>(p.kv) + ((s.k0 + k) * p.H + h) * LAT_KV;
            const T* pe = static_cast<const T*>(p.k_pe) + (s.k0 + k) * p.k_pe_stride;
            float x = 0.f, d = 0.f, kk[6];
            for (int e = 0; e < 6; ++e) kk[e] = to_f(e < 4 ? kv[lane + 32 * e] : pe[lane + 32 * (e - 4)]);
            for (int e = 0; e < 6; ++e) x += qv[e] * kk[e];
            for (int e = 0; e < 4; ++e) d += dv[e] * to_f(kv[LAT_N + lane + 32 * e]);
            x = warp_sum(x);
            d = warp_sum(d);
            const float dx = expf(x - lse) * (d - delta) * p.scale;
            for (int e = 0; e < 6; ++e) acc[e] += dx * kk[e];
        }
        T* out = static_cast<T*>(p.dq) + row * LAT_QK;
        for (int e = 0; e < 6; ++e) out[lane + 32 * e] = from_f<T>(acc[e]);
    }
}

template <typename T>
__global__ void latent_dkv_kernel(LatentParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int n, j;
    latent_slot(p.cu_k, p.Tk, p.N, blockIdx.x, LAT_TILE, n, j);
    LatentSeq s;
    if (!latent_seq(p, n, s)) return;
    const int h = blockIdx.y;
    const long long rows = p.cu_k ? p.Tk : (long long)p.N * p.Tk;
    for (int r = warp; r < LAT_TILE; r += blockDim.x >> 5) {
        const int k = j * LAT_TILE + r;
        if (k >= s.lk) return;
        const T* kv = static_cast<const T*>(p.kv) + ((s.k0 + k) * p.H + h) * LAT_KV;
        const T* pe = static_cast<const T*>(p.k_pe) + (s.k0 + k) * p.k_pe_stride;
        float kk[6], vv[4], dk[6] = {}, dv[4] = {};
        for (int e = 0; e < 6; ++e) kk[e] = to_f(e < 4 ? kv[lane + 32 * e] : pe[lane + 32 * (e - 4)]) * p.scale;
        for (int e = 0; e < 4; ++e) vv[e] = to_f(kv[LAT_N + lane + 32 * e]);
        const int first = p.causal ? max(0, k - (s.lk - s.lq)) : 0;
        for (int i = first; i < s.lq; ++i) {
            const long long row = (s.q0 + i) * p.H + h;
            const T* q = static_cast<const T*>(p.q) + row * LAT_QK;
            const T* dob = static_cast<const T*>(p.dout) + row * LAT_V;
            float x = 0.f, d = 0.f, qv[6], dd[4];
            for (int e = 0; e < 6; ++e) {
                qv[e] = to_f(q[lane + 32 * e]);
                x += qv[e] * kk[e];
            }
            for (int e = 0; e < 4; ++e) {
                dd[e] = to_f(dob[lane + 32 * e]);
                d += dd[e] * vv[e];
            }
            x = warp_sum(x);
            d = warp_sum(d);
            const float w = expf(x - p.lse[row]), dx = w * (d - p.delta[row]) * p.scale;
            for (int e = 0; e < 4; ++e) dv[e] += w * dd[e];
            for (int e = 0; e < 6; ++e) dk[e] += dx * qv[e];
        }
        T* out = static_cast<T*>(p.dkv) + ((s.k0 + k) * p.H + h) * LAT_KV;
        for (int e = 0; e < 4; ++e) {
            out[lane + 32 * e] = from_f<T>(dk[e]);
            out[LAT_N + lane + 32 * e] = from_f<T>(dv[e]);
        }
        float* part = p.dpe_part + ((long long)h * rows + s.k0 + k) * LAT_P;
        for (int e = 0; e < 2; ++e) part[lane + 32 * e] = dk[4 + e];
    }
}

template <typename T>
__global__ void latent_dpe_kernel(LatentParams p, long long rows) {
    const long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (e >= rows * LAT_P) return;
    float sum = 0.f;
    for (int h = 0; h < p.H; ++h) sum += p.dpe_part[h * rows * LAT_P + e];
    static_cast<T*>(p.dk_pe)[e] = from_f<T>(sum);
}

template <typename T>
cudaError_t launch(const LatentParams& p, cudaStream_t stream) {
    const bool varlen = p.cu_q != nullptr;
    const long long rows = varlen ? p.Tk : (long long)p.N * p.Tk;
    if (const int slots = latent_slots(varlen, p.Tq, p.N, LAT_TILE))
        latent_dq_kernel<T><<<dim3(slots, p.H), 256, 0, stream>>>(p);
    if (const int slots = latent_slots(varlen, p.Tk, p.N, LAT_TILE))
        latent_dkv_kernel<T><<<dim3(slots, p.H), 256, 0, stream>>>(p);
    if (rows) latent_dpe_kernel<T><<<(unsigned)((rows * LAT_P + 255) / 256), 256, 0, stream>>>(p, rows);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_latent_bwd(const LatentParams& p, bool fp16, cudaStream_t stream) {
    return fp16 ? launch<__half>(p, stream) : launch<__nv_bfloat16>(p, stream);
}

}  // namespace kda
