// Absorbed latent attention over the paged cache: one warp per (token, head).
#include "kda_latent_decode.cuh"

namespace kda {

namespace {

template <typename T>
__global__ void latent_decode_kernel(DecodeParams p) {
    const int lane = threadIdx.x, h = blockIdx.x, t = blockIdx.y, n = blockIdx.z;
    const long long row = ((long long)n * p.S + t) * p.H + h;
    const T* q = static_cast<const T*>(p.q) + row * LAT_ROW;
    float qv[18], acc[16] = {}, m = -INFINITY, l = 0.f;
    for (int e = 0; e < 18; ++e) qv[e] = to_f(q[lane + 32 * e]) * p.scale;
    const long long most = (long long)p.table_width * p.page_size;
    int len = p.lens[n];
    if (len < 0 || len > most) {
        if (lane == 0) set_status(p.status, STATUS_BAD_PAGE);
        len = len < 0 ? 0 : (int)most;
    }
    const int last = len - p.S + 1 + t;
    for (int k = 0; k < last; ++k) {
        const int page = p.table[(long long)n * p.table_width + k / p.page_size];
        if (page < 0 || page >= p.num_pages) {
            if (lane == 0) set_status(p.status, STATUS_BAD_PAGE);
            continue;
        }
        const T* r = static_cast<const T*>(p.cache) + ((long long)page * p.page_size + k % p.page_size) * LAT_ROW;
        float x = 0.f, rv[18];
        for (int e = 0; e < 18; ++e) {
            rv[e] = to_f(r[lane + 32 * e]);
            x += qv[e] * rv[e];
        }
        x = warp_sum(x);
        const float mn = fmaxf(m, x), c = mn == -INFINITY ? 1.f : expf(m - mn), w = mn == -INFINITY ? 0.f : expf(x - mn);
        l = l * c + w;
        for (int e = 0; e < 16; ++e) acc[e] = acc[e] * c + w * rv[e];
        m = mn;
    }
    T* o = static_cast<T*>(p.o) + row * LAT_C;
    for (int e = 0; e < 16; ++e) o[lane + 32 * e] = from_f<T>(l > 0.f ? acc[e] / l : 0.f);
    if (lane == 0 && p.lse) p.lse[row] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

unsigned long long latent_decode_scratch(int N, int S, int H) { return WS_HEADER; }

cudaError_t launch_latent_decode(const DecodeParams& p, bool fp16, cudaStream_t stream) {
    if (cudaMemsetAsync(p.status, 0, WS_CLEAR, stream) != cudaSuccess) return cudaGetLastError();
    const dim3 grid(p.H, p.S, p.N);
    if (fp16) latent_decode_kernel<__half><<<grid, 32, 0, stream>>>(p);
    else latent_decode_kernel<__nv_bfloat16><<<grid, 32, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace kda
