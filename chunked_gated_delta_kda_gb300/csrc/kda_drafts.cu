// Verification of drafted tokens (kda_verify_drafts), with its C entry point.
// See include/kda.h for the contract.
//
// A cluster of CTAs a sequence.  The drafts are looked at by the first warp of
// each CTA (two gathered numbers a draft), which leaves one position whose
// rows p and q the token behind the drafts is drawn from: the only rows of the
// vocabulary that are read, once.  Every warp sums r = max(p - q, 0) over a
// range of its own; the warps' sums go to all CTAs, and the one whose range
// holds the border u sum r reads that range again and finds the token.
//
// Which token it is depends on the sums' last bits, and 64-bit arithmetic runs
// at two operations a clock and SM here, less than the rows' bytes leave time
// for.  So r and its sums are pairs of 32-bit numbers whose rounding errors are
// kept (Knuth's and Dekker's exact sums): some 2^-46 of the sum, 16 operations
// an element; the warps' sums are joined in 64 bits.
#include <cstdint>

#include "kda.h"
#include "kda_latent_mma.cuh"

namespace kda {

namespace {

constexpr int DR_THREADS = 512;
constexpr int DR_WARPS = DR_THREADS / 32;
constexpr int DR_MOST = 8;                       // CTAs of a cluster
constexpr int DR_SEGS = DR_MOST * DR_WARPS;

struct DraftParams {
    const int64_t* drafts;
    const void* q;                               // or null
    const void* p;
    const float* uniform;
    int64_t* tokens;
    int32_t* accepted;
    uint32_t* status;
    long long q_n, q_s, p_n, p_s;                // strides in elements
    int S, V;
    int seg;                                     // elements of a warp's range, a multiple of 512
};

__device__ __forceinline__ float val(float x) { return x; }
__device__ __forceinline__ float val(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float val(__half x) { return __half2float(x); }

// A sum of non-negative numbers as s + c.
struct Sum {
    float s = 0.f, c = 0.f;
    __device__ __forceinline__ void add(float h, float l) {
        const float t = s + h, b = t - s;
        c += ((s - (t - b)) + (h - b)) + l;
        s = t;
    }
    __device__ __forceinline__ double value() const { return (double)s + (double)c; }
};

// max(p - q, 0) as h + l, exactly; 0 where it is no number.
__device__ __forceinline__ void rest(float p, float q, float& h, float& l) {
    const float d = p - q, b = p - d;
    const bool some = d > 0.f;
    l = some ? (p - (d + b)) + (b - q) : 0.f;
    h = some ? d : 0.f;
}

// How the row r is made: p alone, p - q, or p without one token.
enum Kind { P_ALONE, P_LESS_Q, P_BUT_ONE };

template <typename T>
struct Row {
    const T* p;
    const T* q;
    Kind kind;
    int but;
    __device__ __forceinline__ void weigh(int i, float x, float y, float& h, float& l) const {
        rest(x, kind == P_LESS_Q ? y : 0.f, h, l);
        if (kind == P_BUT_ONE && i == but) h = l = 0.f;
    }
    __device__ __forceinline__ void at(int i, float& h, float& l) const {
        weigh(i, val(__ldg(p + i)), kind == P_LESS_Q ? val(__ldg(q + i)) : 0.f, h, l);
    }
};

// The sum of [from, to), whole warp, in every lane.  VEC: the rows start on 16
// bytes, and so does `from`.
template <typename T, bool VEC>
__device__ __forceinline__ double sum_range(const Row<T>& row, int from, int to) {
    constexpr int W = VEC ? 16 / (int)sizeof(T) : 1, BATCH = VEC ? 16 / W : 8;   // (512 elements of a warp at a time)
    const int lane = threadIdx.x & 31;
    Sum sum;
    int i = from + lane * W;
    union Piece {
        uint4 u;
        T t[16 / sizeof(T)];
    };
    for (; i + (BATCH - 1) * 32 * W + W <= to; i += BATCH * 32 * W) {
        Piece x[BATCH], y[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            if constexpr (VEC) x[k].u = __ldg(reinterpret_cast<const uint4*>(row.p + i + k * 32 * W));
            else x[k].t[0] = row.p[i + k * 32];
        }
        if (row.kind == P_LESS_Q) {
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                if constexpr (VEC) y[k].u = __ldg(reinterpret_cast<const uint4*>(row.q + i + k * 32 * W));
                else y[k].t[0] = row.q[i + k * 32];
            }
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
#pragma unroll
            for (int e = 0; e < W; ++e) {
                float h, l;
                row.weigh(i + k * 32 * W + e, val(x[k].t[e]), row.kind == P_LESS_Q ? val(y[k].t[e]) : 0.f, h, l);
                sum.add(h, l);
            }
    }
    for (; i < to; i += 32 * W) {
#pragma unroll
        for (int e = 0; e < W; ++e)
            if (i + e < to) {
                float h, l;
                row.at(i + e, h, l);
                sum.add(h, l);
            }
    }
    double d = sum.value();
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) d += __shfl_xor_sync(0xffffffffu, d, m);
    return d;
}

// Inclusive prefix sum over the lanes.
__device__ __forceinline__ double lanes_upto(double x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    return x;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(DR_THREADS, 2) verify_drafts_kernel(const __grid_constant__ DraftParams p) {
    __shared__ double sums[2][DR_SEGS], parts[DR_THREADS];
    __shared__ double bound;
    __shared__ int taken_s, drafted_s, seg_s, best_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank(), n = blockIdx.x / ctas;
    const int64_t* drafts = p.drafts + (long long)n * p.S;
    const T* target = static_cast<const T*>(p.p) + n * p.p_n;
    const T* draft = p.q ? static_cast<const T*>(p.q) + n * p.q_n : nullptr;
    const float* uniform = p.uniform + (long long)n * (p.S + 1);

    if (warp == 0) {
        int taken = 0, drafted = 0;              // accepted; whether the one behind them is a draft
        bool bad = false;
        for (int base = 0; base < p.S; base += 32) {
            const int s = base + lane;
            const int64_t d = s < p.S ? drafts[s] : -1;
            const bool there = d >= 0 && d < p.V;
            bad |= d >= p.V;
            bool yes = false;
            if (there) {
                const double x = val(target[s * p.p_s + d]), y = draft ? val(draft[s * p.q_s + d]) : 1.0;
                yes = (double)uniform[s] * y < x;    // exact: 24 bits times 24
            }
            const uint32_t no = ~__ballot_sync(0xffffffffu, yes), is = __ballot_sync(0xffffffffu, there);
            taken += no ? __ffs(no) - 1 : 32;
            if (no) {
                drafted = (is >> (__ffs(no) - 1)) & 1u;
                // a token past the vocabulary counts where the drafts before it were accepted
                bad = bad && lane <= __ffs(no) - 1;
                break;
            }
        }
        if (bad && rank == 0) set_status(p.status, STATUS_BAD_TOKEN);
        if (lane == 0) taken_s = taken, drafted_s = drafted;
    }
    __syncthreads();
    const int taken = taken_s;
    if (rank == 0) {
        for (int s = tid; s <= p.S; s += DR_THREADS)
            if (s != taken) p.tokens[(long long)n * (p.S + 1) + s] = s < taken ? drafts[s] : -1;
        if (tid == 0) p.accepted[n] = taken + 1;
    }
    Row<T> row;
    row.p = target + taken * p.p_s;
    row.q = draft ? draft + taken * p.q_s : nullptr;
    row.kind = !drafted_s ? P_ALONE : draft ? P_LESS_Q : P_BUT_ONE;
    row.but = row.kind == P_BUT_ONE ? (int)drafts[taken] : -1;
    const double u = uniform[p.S];

    const int segs = ctas * DR_WARPS, mine = rank * DR_WARPS + warp;
    double total = 0.0;
    int round = 0;
    cluster_barrier();                           // every CTA's shared memory is there
    for (;; ++round) {
        const int from = min((long long)p.V, (long long)mine * p.seg), to = min((long long)p.V, (long long)from + p.seg);
        const double d = sum_range<T, VEC>(row, from, to);
        if (lane < ctas) {
            const uint32_t at = cluster_addr(smem_u32(&sums[round][mine]), lane);
            asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(at), "d"(d) : "memory");
        }
        cluster_barrier();
        if (warp == 0) {
            // the range that holds the border: the first whose sums up to it are above, else the last with weight
            double up[DR_SEGS / 32], x[DR_SEGS / 32], all = 0.0;
#pragma unroll
            for (int k = 0; k < DR_SEGS / 32; ++k) {
                const int s = 32 * k + lane;
                x[k] = s < segs ? sums[round][s] : 0.0;
                up[k] = lanes_upto(x[k]) + all;
                all = __shfl_sync(0xffffffffu, up[k], 31);
            }
            const double border = u * all;
            int seg = -1, last = -1;
            double before = 0.0;
#pragma unroll
            for (int k = 0; k < DR_SEGS / 32; ++k) {
                const uint32_t above = __ballot_sync(0xffffffffu, x[k] > 0.0 && up[k] > border);
                const uint32_t some = __ballot_sync(0xffffffffu, x[k] > 0.0);
                if (some) last = 32 * k + 31 - __clz(some);
                if (seg < 0 && above) {
                    seg = 32 * k + __ffs(above) - 1;
                    before = __shfl_sync(0xffffffffu, up[k] - x[k], __ffs(above) - 1);
                }
            }
            if (lane == 0) {
                seg_s = seg >= 0 ? seg : last;
                bound = seg >= 0 ? border - before : INFINITY;
                parts[0] = all;
                best_s = -1;
            }
        }
        __syncthreads();
        total = parts[0];
        if (total > 0.0 || row.kind == P_ALONE || round == 1) break;
        row.kind = P_ALONE;                      // p = q everywhere: p itself
    }
    const int seg = seg_s;
    const bool fine = total > 0.0 && total < INFINITY && seg >= 0;
    if (!fine) {
        if (rank == 0 && tid == 0) {
            p.tokens[(long long)n * (p.S + 1) + taken] = 0;
            set_status(p.status, STATUS_BAD_TOKEN);
        }
        return;
    }
    if (seg / DR_WARPS != rank) return;
    // this CTA's range: a thread a run of elements, then the run that holds the border
    const int from = seg * p.seg, to = min((long long)p.V, (long long)from + p.seg);
    const int each = p.seg / DR_THREADS, a = min(to, from + tid * each), b = min(to, a + each);
    Sum sum;
    for (int i = a; i < b; ++i) {
        float h, l;
        row.at(i, h, l);
        sum.add(h, l);
    }
    const double own = sum.value(), upto = lanes_upto(own);
    __syncthreads();                             // parts[0] has been read
    if (lane == 31) parts[warp] = upto;
    __syncthreads();
    double before = 0.0;
    for (int w = 0; w < warp; ++w) before += parts[w];
    const bool some = own > 0.0, above = some && before + upto > bound;
    // the first run above the border, else the last with weight
    const int first_above = __reduce_min_sync(0xffffffffu, above ? tid : DR_THREADS);
    const int last_some = __reduce_max_sync(0xffffffffu, some ? tid : -1);
    __shared__ int firsts[DR_WARPS], lasts[DR_WARPS];
    if (lane == 0) firsts[warp] = first_above, lasts[warp] = last_some;
    __syncthreads();
    int run = DR_THREADS, last = -1;
    for (int w = 0; w < DR_WARPS; ++w) run = min(run, firsts[w]), last = max(last, lasts[w]);
    const bool found = run < DR_THREADS;
    if (!found) run = last;
    if (tid != run) return;
    double c = before + (upto - own);
    int token = a;
    for (int i = a; i < b; ++i) {
        float h, l;
        row.at(i, h, l);
        if (h > 0.f) {
            token = i;
            c += (double)h + (double)l;
            if (found && c > bound) break;
        }
    }
    p.tokens[(long long)n * (p.S + 1) + taken] = token;
}

template <typename T>
cudaError_t launch(const DraftParams& p, bool vec, int N, int ctas, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(N * ctas));
    cfg.blockDim = dim3(DR_THREADS);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return vec ? cudaLaunchKernelEx(&cfg, verify_drafts_kernel<T, true>, p) : cudaLaunchKernelEx(&cfg, verify_drafts_kernel<T, false>, p);
}

bool off(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

}  // namespace

}  // namespace kda

extern "C" kda_status kda_verify_drafts(const int64_t* draft_tokens, const void* draft_probs, const long long* draft_strides,
                                        const void* target_probs, const long long* target_strides, const float* uniform,
                                        int64_t* tokens, int32_t* num_accepted, int N, int S, int V, unsigned flags,
                                        void* workspace, cudaStream_t stream) {
    using namespace kda;
    if (N < 1 || S < 0 || V < 1 || N > (1 << 24) || V > (1 << 30) || S == INT32_MAX) return KDA_ERR_INVALID_ARG;
    if ((flags & ~(KDA_FLAG_FP16 | KDA_FLAG_FP32)) != 0u || flags == (KDA_FLAG_FP16 | KDA_FLAG_FP32)) return KDA_ERR_INVALID_ARG;
    if ((S > 0 && !draft_tokens) || !target_probs || !target_strides || !uniform || !tokens || !num_accepted ||
        (draft_probs && !draft_strides))
        return KDA_ERR_INVALID_ARG;
    const unsigned size = (flags & KDA_FLAG_FP32) != 0u ? 4u : 2u;
    if (off(draft_tokens, 8) || off(draft_probs, size) || off(target_probs, size) || off(uniform, 4) || off(tokens, 8) ||
        off(num_accepted, 4) || off(workspace, 256))
        return KDA_ERR_INVALID_ARG;
    DraftParams p{};
    p.drafts = draft_tokens, p.q = draft_probs, p.p = target_probs, p.uniform = uniform;
    p.tokens = tokens, p.accepted = num_accepted, p.status = static_cast<uint32_t*>(workspace);
    p.p_n = target_strides[0], p.p_s = target_strides[1];
    if (draft_probs) p.q_n = draft_strides[0], p.q_s = draft_strides[1];
    p.S = S, p.V = V;
    const long long most = 1ll << 40;
    for (const long long x : {p.p_n, p.p_s, p.q_n, p.q_s})
        if (x < 0 || x >= most) return KDA_ERR_INVALID_ARG;
    const long long pieces = 16 / size;
    const bool vec = !off(target_probs, 16) && !off(draft_probs, 16) && p.p_n % pieces == 0 && p.p_s % pieces == 0 &&
                     p.q_n % pieces == 0 && p.q_s % pieces == 0;
    // as many CTAs a sequence as fit the GPU at once (two an SM), and have 512 elements a warp
    int ctas = 1;
    while (ctas < DR_MOST && (long long)ctas * DR_WARPS * 512 < V && 2ll * ctas * N <= 304) ctas *= 2;
    p.seg = (int)(((long long)V + ctas * DR_WARPS * 512 - 1) / (ctas * DR_WARPS * 512) * 512);
    if (p.status && cudaMemsetAsync(p.status, 0, WS_CLEAR, stream) != cudaSuccess) return KDA_ERR_CUDA;
    const cudaError_t e = (flags & KDA_FLAG_FP32) != 0u   ? launch<float>(p, vec, N, ctas, stream)
                          : (flags & KDA_FLAG_FP16) != 0u ? launch<__half>(p, vec, N, ctas, stream)
                                                          : launch<__nv_bfloat16>(p, vec, N, ctas, stream);
    return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
