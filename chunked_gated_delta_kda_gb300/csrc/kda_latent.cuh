// Shared definitions of the latent-attention kernels: sizes, parameters, the
// map from 128-row tile slots to sequences, and the 16-bit float types.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kda_common.cuh"

namespace kda {

constexpr int LAT_C = 512;                  // latent channels of a cached row
constexpr int LAT_P = 64;                   // positional channels, shared by the heads
constexpr int LAT_ROW = LAT_C + LAT_P;      // a cached row, an absorbed query
constexpr int LAT_N = 128;                  // per-head key channels (expanded)
constexpr int LAT_V = 128;                  // value channels (expanded)
constexpr int LAT_QK = LAT_N + LAT_P;       // expanded query
constexpr int LAT_KV = LAT_N + LAT_V;       // expanded key and value of one token and head
constexpr int LAT_TILE = 128;               // rows of a query or key tile

constexpr int LATENT_SHARE_ITEMS = 896;     // records of shared key ranges in the forward's workspace

struct LatentParams {
    const void* q;          // [B*Tq, H, 192]
    const void* kv;         // [B*Tk, H, 256]
    const void* k_pe;       // [B*Tk, 64], k_pe_stride elements apart
    long long k_pe_stride;
    const void* o;          // backward: [B*Tq, H, 128]
    const float* lse;       // backward: [B*Tq, H]
    const void* dout;       // backward: [B*Tq, H, 128]
    void* o_out;            // forward
    float* lse_out;         // forward, or null
    void* dq;
    void* dkv;
    void* dk_pe;
    float* aux;             // backward workspace: per (64-query tile slot, head) 64 log2 lse, 64 dout . o
    int4* share_items;      // forward's workspace for shared key ranges (see there), or null
    float* share_parts;
    float* dpe_part;        // backward workspace: [H][B*Tk][64] per-head gradients of k_pe
    const int32_t* cu_q;    // int32 [N+1] or null
    const int32_t* cu_k;
    uint32_t* status;       // or null
    float scale;
    int Tq, Tk;             // per sequence (fixed) or packed (varlen)
    int H, N;
    int causal;
    uint32_t wait_limit;
};

// A sequence's queries [q0, q0 + lq) and keys [k0, k0 + lk) as packed rows.
struct LatentSeq {
    long long q0, k0;
    int lq, lk;
};

__device__ __forceinline__ void set_status(uint32_t* status, uint32_t bit) {
    if (status != nullptr) atomicOr(status, bit);
}

// False (and the status word flagged) where the offsets are not a valid
// non-decreasing list into [0, T].
__device__ __forceinline__ bool latent_seq(const LatentParams& p, int n, LatentSeq& s) {
    if (p.cu_q == nullptr) {
        s.q0 = (long long)n * p.Tq;
        s.k0 = (long long)n * p.Tk;
        s.lq = p.Tq;
        s.lk = p.Tk;
        return true;
    }
    const int a = p.cu_q[n], b = p.cu_q[n + 1], c = p.cu_k[n], d = p.cu_k[n + 1];
    if (a < 0 || b < a || b > p.Tq || (n == 0 && a != 0) || (n == p.N - 1 && b != p.Tq) || c < 0 || d < c ||
        d > p.Tk || (n == 0 && c != 0) || (n == p.N - 1 && d != p.Tk)) {
        set_status(p.status, STATUS_BAD_CU);
        return false;
    }
    s.q0 = a;
    s.k0 = c;
    s.lq = b - a;
    s.lk = d - c;
    return true;
}

// A decreasing step in either list, looked for by `threads` threads: the tile
// slots of a list that is not sorted can pass over a sequence (0, 600, 300, 900
// with tiles of 256: its second), whose offsets latent_seq then never sees.
__device__ __forceinline__ void check_offsets(const LatentParams& p, int t, int threads) {
    if (p.cu_q == nullptr || p.status == nullptr) return;
    bool bad = false;
    for (int n = t; n < p.N; n += threads) bad |= p.cu_q[n + 1] < p.cu_q[n] || p.cu_k[n + 1] < p.cu_k[n];
    if (bad) set_status(p.status, STATUS_BAD_CU);
}

// Tile slots over packed rows with offsets cu (null: N sequences of T rows),
// `tile` rows each: slot floor(cu[n] / tile) + n + j holds tile j of sequence
// n, so floor(T / tile) + N slots hold every tile and some hold none.
__host__ __device__ __forceinline__ int latent_slots(bool varlen, int T, int N, int tile) {
    return varlen ? T / tile + N : N * ((T + tile - 1) / tile);
}

__device__ __forceinline__ void latent_slot(const int32_t* cu, int T, int N, int slot, int tile, int& n, int& j) {
    if (cu == nullptr) {
        const int per = (T + tile - 1) / tile;
        n = slot / per;
        j = slot % per;
        return;
    }
    int lo = 0, hi = N - 1;   // the last n with floor(cu[n] / tile) + n <= slot
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] / tile + mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    n = lo;
    j = slot - (cu[lo] / tile + lo);
}

// The sequence and tile of a slot, whole warp: the offsets of up to 31 packed
// sequences in one round of loads (a bisection is a chain of them, 2000 cycles
// at the start of a CTA).  The sequence comes out of a vote and its offsets
// are loaded again from there: values from a vote or a uniform load stay
// uniform for the compiler, those from a shuffle do not, and every product
// that depends on one costs several times as much.  (For the same reason the
// kernels search before their first inline assembly: behind it, forward and
// backward took 6 % longer.)  `cu` is p.cu_q or p.cu_k.
__device__ __forceinline__ bool latent_find(const LatentParams& p, const int32_t* cu, int T, int slot, int tile, int& n, int& j,
                                            LatentSeq& s) {
    if (cu == nullptr || p.N > 31) {
        latent_slot(cu, T, p.N, slot, tile, n, j);
        return latent_seq(p, n, s);
    }
    const int lane = threadIdx.x & 31;
    const int first = lane < p.N ? cu[lane] : INT32_MAX / 2;
    const uint32_t le = __ballot_sync(0xffffffffu, first / tile + lane <= slot);
    n = le != 0u ? 31 - __clz(le) : 0;
    if (!latent_seq(p, n, s)) return false;
    j = slot - (int)((cu == p.cu_q ? s.q0 : s.k0) / tile + n);
    return true;
}

// Launch order.  CTAs start in the order of their index and differ in work, so
// a sequence's largest tiles come first (its last ones where `last`), all heads
// of a tile next to each other.  Heads after one another, which keeps fewer
// keys in use at a time, was slower wherever the last head's large tiles came
// late (forward / backward, us, a few calls at a time: T=8192 H=8 170 / 492 ->
// 117 / 422, packed T=9192 H=32 258 / 939 -> 228 / 888, B=4 T=8192 H=16 880 /
// 3408 -> 828 / 3391; 32 packed sequences of 2048, H=16, 622 / 2372 -> 600 /
// 2419); the tiles of all sequences of equal length by size was slower as well
// (B=8 T=2048 H=16 171 / 650 beside 150 / 588).
__device__ __forceinline__ void latent_order(const LatentParams& p, int index, int slots, bool last, int& slot, int& h) {
    const int at = index / p.H;
    h = index - at * p.H;
    slot = last ? slots - 1 - at : at;
}

// ---- 16-bit floats ----
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

}  // namespace kda
