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
// for.  So r, its sums and the border are pairs of 32-bit numbers whose
// rounding errors are kept (Knuth's and Dekker's exact sums), two elements an
// operation: ten for an element, four without q.  The errors' own sum has 32
// bits too, so after 128 additions in a thread (a vocabulary of 2^17 and more)
// it all goes into a pair in shared memory, which takes no registers from the
// loads (kept in registers: 128 x 131072 4 % slower).  n additions are off by
// n^2 2^-48 of their sum at most, a chain of m pairs by 3 m 2^-48, the border
// by 2^-31 of the total at V = 2^30: less than u can tell apart.  (A replay of
// 2^18 additions: exponentials of uniform numbers 2^-43, one number again and
// again 0; without the pairs 2^-29 and 2^-18.)
//
// In a graph: 128 sequences of 131072 in fp32 (134 MB) 21.7 us, 6.2 TB/s (26.5
// called one by one), 256 of them 41, 6.6 (with sums in 64 bits where warps join
// 31, one element an operation 23).  One sequence of 32768: 6.6 us: the launch,
// the drafts' two rounds of loads, the row's, the cluster's exchange and the last
// range's, about one each.  Rows of odd length start anywhere: the warps' ranges
// begin on 16 bytes of p, and q's words are shifted together (256 x 50257 in bf16
// without q 12.5 us; element by element 28).  16-bit rows with q are bound by
// their operations (256 x 65536: 18.5 us, 3.6 TB/s).
#include <cstdint>
#include <type_traits>

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

// A number as h + l, l what h lost in rounding.
struct Pair {
    float h, l;
};
__device__ __forceinline__ Pair pair_of(float s, float c) {      // |s| not below |c|, or s = 0
    const float h = s + c;
    return {h, c - (h - s)};
}
__device__ __forceinline__ Pair operator+(Pair x, Pair y) {
    const float s = x.h + y.h, b = s - x.h;
    return pair_of(s, ((x.h - (s - b)) + (y.h - b)) + (x.l + y.l));
}
__device__ __forceinline__ Pair operator-(Pair x, Pair y) { return x + Pair{-y.h, -y.l}; }
__device__ __forceinline__ Pair operator*(float u, Pair x) {
    const float p = u * x.h;
    return pair_of(p, fmaf(u, x.h, -p) + u * x.l);
}
__device__ __forceinline__ bool operator>(Pair x, Pair y) { return x.h > y.h || (x.h == y.h && x.l > y.l); }
template <typename SHFL>
__device__ __forceinline__ Pair moved(Pair x, SHFL f) {
    return {f(x.h), f(x.l)};
}

// A sum of non-negative numbers as s + c.
struct Sum {
    float s = 0.f, c = 0.f;
    __device__ __forceinline__ void add(float h, float l) {
        const float t = s + h, b = t - s;
        c += ((s - (t - b)) + (h - b)) + l;
        s = t;
    }
    __device__ __forceinline__ Pair value() const { return pair_of(s, c); }
};

// Two 32-bit numbers an operation (the sums of even and of odd elements).
using Two = unsigned long long;
__device__ __forceinline__ Two two(float a, float b) {
    Two x;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
    return x;
}
__device__ __forceinline__ float2 halves(Two x) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(x));
    return v;
}
__device__ __forceinline__ Two plus(Two a, Two b) {
    Two x;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(a), "l"(b));
    return x;
}
__device__ __forceinline__ Two minus(Two a, Two b) {
    Two x;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(x) : "l"(b), "l"(0xbf800000bf800000ull), "l"(a));
    return x;
}
struct TwoSums {
    Two s = 0, c = 0;
    __device__ __forceinline__ void add(Two h) {
        const Two t = plus(s, h), b = minus(t, s);
        c = plus(c, plus(minus(s, minus(t, b)), minus(h, b)));
        s = t;
    }
    // max(p - q, 0), as rest() below
    __device__ __forceinline__ void add_rest(Two p, Two q) {
        const Two d = minus(p, q), b = minus(p, d);
        const float2 h = halves(d), l = halves(plus(minus(p, plus(d, b)), minus(b, q)));
        add(two(h.x > 0.f ? h.x : 0.f, h.y > 0.f ? h.y : 0.f));
        c = plus(c, two(h.x > 0.f ? l.x : 0.f, h.y > 0.f ? l.y : 0.f));
    }
    __device__ __forceinline__ Pair value() const {
        const float2 x = halves(s), y = halves(c);
        return pair_of(x.x, y.x) + pair_of(x.y, y.y);
    }
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
    int but;                                     // -1 where no token is left out
    __device__ __forceinline__ void at(int i, float& h, float& l) const {
        rest(val(__ldg(p + i)), kind == P_LESS_Q ? val(__ldg(q + i)) : 0.f, h, l);
        if (i == but) h = l = 0.f;
    }
};

// 16 bytes of elements.
template <typename T>
union Piece {
    uint4 u;
    T t[16 / sizeof(T)];
};

// Elements 2 j and 2 j + 1 of them.
template <typename T>
__device__ __forceinline__ float2 pair_at(uint4 u, int j) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
    else return unpack2<sizeof(T) == 2 && !std::is_same<T, __nv_bfloat16>::value>(w[j]);
}

// A whole 16-byte word of a row [begin, end), 0 where the row is not.
template <typename T>
__device__ __forceinline__ uint4 load_word(const uint4* word, const T* begin, const T* end) {
    const T* at = reinterpret_cast<const T*>(word);
    constexpr int W = 16 / (int)sizeof(T);
    if (at >= begin && end - at >= W) return __ldg(word);
    Piece<T> x;
    x.u = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < W; ++e)
        if (at + e >= begin && at + e < end) x.t[e] = at[e];
    return x.u;
}

// 16 bytes of a row from any element on, a lane the next ones: the words that
// they lie in, whose second the next lane has loaded as its first.  EDGE: they
// may reach past the row, where they are 0.
template <bool EDGE, typename T>
__device__ __forceinline__ uint4 load_any(const T* at, const T* begin, const T* end) {
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(at) & 15u);
    const uint4* words = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(at) & ~(uintptr_t)15u);
    const uint4 x = EDGE ? load_word(words, begin, end) : __ldg(words);
    if (off == 0) return x;                      // all lanes alike
    uint4 y = x;
    if ((threadIdx.x & 31) == 31) y = EDGE ? load_word(words + 1, begin, end) : __ldg(words + 1);
    const int from = ((threadIdx.x & 31) + 1) & 31;
    const uint4 z = make_uint4(__shfl_sync(0xffffffffu, x.x, from), __shfl_sync(0xffffffffu, x.y, from), __shfl_sync(0xffffffffu, x.z, from),
                               __shfl_sync(0xffffffffu, x.w, from));
    if ((threadIdx.x & 31) != 31) y = z;
    uint32_t w[6] = {x.x, x.y, x.z, x.w, y.x, y.y};
    if (off & 8u) w[0] = w[2], w[1] = w[3], w[2] = w[4], w[3] = w[5], w[4] = y.z, w[5] = y.w;
    if (off & 4u) w[0] = w[1], w[1] = w[2], w[2] = w[3], w[3] = w[4], w[4] = w[5];
    const uint32_t bits = 8u * (off & 3u);
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                      __funnelshift_r(w[3], w[4], bits));
}

template <int N>
struct Number {
    static constexpr int value = N;
};

// The sum of [from, to) of a row of V, whole warp, in every lane; row.p + from
// is on 16 bytes (`from` may be below 0: what is in front of the row counts
// nothing), `to` is V or `from` and a multiple of 512.  LESS: of p - q, whose
// rows start on 16 bytes where p's do if ALIGNED, and anywhere if not.
// `carried` is the thread's own.
template <typename T, bool ALIGNED, bool LESS>
__device__ __forceinline__ Pair sum_range(const Row<T>& row, int from, int to, int V, Pair* carried) {
    constexpr int W = 16 / (int)sizeof(T);
    const int lane = threadIdx.x & 31;
    TwoSums sums;
    // BATCH x 32 pieces of 16 bytes from element i on
    auto chunk = [&](auto batch, auto edge, int i) {
        constexpr int BATCH = decltype(batch)::value;
        constexpr bool EDGE = decltype(edge)::value != 0;
        Piece<T> x[BATCH];
        [[maybe_unused]] Piece<T> y[LESS ? BATCH : 1];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const uint4* at = reinterpret_cast<const uint4*>(row.p + i + (k * 32 + lane) * W);
            if constexpr (EDGE) x[k].u = load_word(at, row.p, row.p + V);
            else x[k].u = __ldg(at);
        }
        if constexpr (LESS) {
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const T* at = row.q + i + (k * 32 + lane) * W;
                if constexpr (ALIGNED && !EDGE) y[k].u = __ldg(reinterpret_cast<const uint4*>(at));
                else y[k].u = load_any<EDGE>(at, row.q, row.q + V);
            }
        }
        if constexpr (EDGE && !LESS) {
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int left_out = row.but - i - (k * 32 + lane) * W;
                if (left_out >= 0 && left_out < W) {
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        if (e == left_out) x[k].t[e] = T(0.f);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
#pragma unroll
            for (int j = 0; j < W / 2; ++j) {
                const float2 a = pair_at<T>(x[k].u, j);
                if constexpr (LESS) {
                    const float2 b = pair_at<T>(y[k].u, j);
                    sums.add_rest(two(a.x, a.y), two(b.x, b.y));
                } else {
                    sums.add(two(fmaxf(a.x, 0.f), fmaxf(a.y, 0.f)));   // (0 from what is no number)
                }
            }
    };
    // whole steps, where they neither reach past the row nor hold the token that is left out
    constexpr int MOST = W == 8 ? 4 : LESS ? 4 : 8, STEP = 32 * W * MOST, HALF = 512 / (32 * W), CARRY = 8;
    auto plain = [&](int i, int count) {
        if constexpr (LESS) return i >= (ALIGNED ? 0 : W) && i + count <= to && (ALIGNED || i + count + W <= V);
        else return i >= 0 && i + count <= to && (row.but < i || row.but >= i + count);
    };
    int i = from, steps = 0;
    while (i < to) {
        for (; plain(i, STEP); i += STEP) {
            chunk(Number<MOST>(), Number<0>(), i);
            if (++steps % CARRY == 0) {
                *carried = steps == CARRY ? sums.value() : *carried + sums.value();
                sums = TwoSums();
            }
        }
        for (; plain(i, 512); i += 512) chunk(Number<HALF>(), Number<0>(), i);
        if (i < to) chunk(Number<1>(), Number<1>(), i);
        i += 32 * W;
    }
    Pair d = sums.value();
    if (steps >= CARRY) d = *carried + d;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) d = d + moved(d, [&](float x) { return __shfl_xor_sync(0xffffffffu, x, m); });
    return d;
}

// Inclusive prefix sum over the lanes.
__device__ __forceinline__ Pair lanes_upto(Pair x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Pair y = moved(x, [&](float z) { return __shfl_up_sync(0xffffffffu, z, d); });
        if (lane >= d) x = y + x;
    }
    return x;
}

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(DR_THREADS, 2) verify_drafts_kernel(const __grid_constant__ DraftParams p) {
    __shared__ Pair sums[2][DR_SEGS], parts[DR_WARPS], bound_s, total_s;
    __shared__ Pair carried[DR_THREADS];
    __shared__ int taken_s, drafted_s, seg_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ctas = (int)cluster_size(), rank = (int)cluster_rank(), n = blockIdx.x / ctas;
    const int64_t* drafts = p.drafts + (long long)n * p.S;
    const T* target = static_cast<const T*>(p.p) + n * p.p_n;
    const T* draft = p.q ? static_cast<const T*>(p.q) + n * p.q_n : nullptr;
    const float* uniform = p.uniform + (long long)n * (p.S + 1);

    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
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
    const float u = uniform[p.S];
    const int shift = (int)((reinterpret_cast<uintptr_t>(row.p) & 15u) / sizeof(T));   // ranges begin on 16 bytes

    const int segs = ctas * DR_WARPS, mine = rank * DR_WARPS + warp;
    Pair total;
    cluster_barrier();                           // every CTA's shared memory is there
    for (int round = 0;; ++round) {
        const int from = (int)min((long long)p.V, (long long)mine * p.seg - shift), to = (int)min((long long)p.V, (long long)from + p.seg);
        const Pair d = row.kind == P_LESS_Q ? sum_range<T, ALIGNED, true>(row, from, to, p.V, carried + tid)
                                            : sum_range<T, ALIGNED, false>(row, from, to, p.V, carried + tid);
        if (lane < ctas) {
            const uint32_t at = cluster_addr(smem_u32(&sums[round][mine]), lane);
            asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(d.h), "f"(d.l) : "memory");
        }
        cluster_barrier();
        if (warp == 0) {
            // the range that holds the border: the first whose sums up to it are above, else the last with weight; a lane PER
            // ranges in a row
            constexpr int PER = DR_SEGS / 32;
            Pair x[PER], up[PER];
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                x[k] = PER * lane + k < segs ? sums[round][PER * lane + k] : Pair{0.f, 0.f};
                up[k] = k == 0 ? x[0] : up[k - 1] + x[k];
            }
            const Pair lanes = lanes_upto(up[PER - 1]), all = moved(lanes, [&](float z) { return __shfl_sync(0xffffffffu, z, 31); });
            Pair ahead = moved(lanes, [&](float z) { return __shfl_up_sync(0xffffffffu, z, 1); });
            if (lane == 0) ahead = {0.f, 0.f};
            const Pair border = u * all;
            int first = -1, weight = -1;
            Pair before = {0.f, 0.f};
#pragma unroll
            for (int k = PER - 1; k >= 0; --k) {
                if (!(x[k].h > 0.f)) continue;
                if (weight < 0) weight = PER * lane + k;
                if (ahead + up[k] > border) {
                    first = PER * lane + k;
                    before = k == 0 ? ahead : ahead + up[k - 1];
                }
            }
            const uint32_t above = __ballot_sync(0xffffffffu, first >= 0);
            const int last = __reduce_max_sync(0xffffffffu, weight);
            const int at = above ? __ffs(above) - 1 : 0, seg = __shfl_sync(0xffffffffu, first, at);
            before = moved(before, [&](float z) { return __shfl_sync(0xffffffffu, z, at); });
            if (lane == 0) {
                seg_s = seg >= 0 ? seg : last;
                bound_s = seg >= 0 ? border - before : Pair{INFINITY, 0.f};
                total_s = all;
            }
        }
        __syncthreads();
        total = total_s;
        if (total.h > 0.f || row.kind == P_ALONE || round == 1) break;
        row.kind = P_ALONE;                      // p = q everywhere: p itself
        row.but = -1;
    }
    const int seg = seg_s;
    if (!(total.h > 0.f && total.h < INFINITY && seg >= 0)) {
        if (rank == 0 && tid == 0) {
            p.tokens[(long long)n * (p.S + 1) + taken] = 0;
            set_status(p.status, STATUS_BAD_TOKEN);
        }
        return;
    }
    if (seg / DR_WARPS != rank) return;
    // this CTA's range: a thread a run of elements, then the run that holds the border, a lane an element
    const Pair bound = bound_s;
    const int from = seg * p.seg - shift, to = (int)min((long long)p.V, (long long)from + p.seg);
    const int each = p.seg / DR_THREADS, a = max(0, min(to, from + tid * each)), b = max(0, min(to, from + (tid + 1) * each));
    auto some = [&](int first, int last) {
        Sum sum;
#pragma unroll 8
        for (int i = first; i < last; ++i) {
            float h, l;
            row.at(i, h, l);
            sum.add(h, l);
        }
        return sum.value();
    };
    Pair own = some(a, min(b, a + 64));
    for (int i = a + 64; i < b; i += 64) own = own + some(i, min(b, i + 64));
    const Pair upto = lanes_upto(own);
    if (lane == 31) parts[warp] = upto;
    __syncthreads();
    // the first warp whose runs reach above the border, else the last with weight; all others are done
    const Pair part = lane < DR_WARPS ? parts[lane] : Pair{0.f, 0.f}, parts_upto = lanes_upto(part);
    const uint32_t over_warps = __ballot_sync(0xffffffffu, part.h > 0.f && parts_upto > bound);
    const uint32_t with_weight = __ballot_sync(0xffffffffu, part.h > 0.f);
    if (warp != (over_warps ? __ffs(over_warps) - 1 : max(0, 31 - __clz(with_weight)))) return;
    const Pair before = moved(parts_upto - part, [&](float z) { return __shfl_sync(0xffffffffu, z, warp); });
    const uint32_t over_runs = __ballot_sync(0xffffffffu, own.h > 0.f && before + upto > bound), runs = __ballot_sync(0xffffffffu, own.h > 0.f);
    const int run = warp * 32 + (over_runs ? __ffs(over_runs) - 1 : max(0, 31 - __clz(runs)));
    Pair c = moved(before + (upto - own), [&](float z) { return __shfl_sync(0xffffffffu, z, run & 31); });
    const int a0 = max(0, min(to, from + run * each)), b0 = max(0, min(to, from + (run + 1) * each));
    int token = -1, latest = a0;                 // (a sum's last bits may put the border behind its run: the last with weight then)
    for (int base = a0; base < b0 && token < 0; base += 32) {
        float h = 0.f, l = 0.f;
        if (base + lane < b0) row.at(base + lane, h, l);
        const Pair up = c + lanes_upto(pair_of(h, l));
        const uint32_t weights = __ballot_sync(0xffffffffu, h > 0.f), over = __ballot_sync(0xffffffffu, h > 0.f && up > bound);
        if (over) token = base + __ffs(over) - 1;
        if (weights) latest = base + 31 - __clz(weights);
        c = moved(up, [&](float z) { return __shfl_sync(0xffffffffu, z, 31); });
    }
    if (lane == 0) p.tokens[(long long)n * (p.S + 1) + taken] = token >= 0 ? token : latest;
}

template <typename T>
cudaError_t launch(const DraftParams& p, bool aligned, int N, int ctas, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // set up beside the kernel before, which it waits for
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(N * ctas));
    cfg.blockDim = dim3(DR_THREADS);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return aligned ? cudaLaunchKernelEx(&cfg, verify_drafts_kernel<T, true>, p) : cudaLaunchKernelEx(&cfg, verify_drafts_kernel<T, false>, p);
}

bool off(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

}  // namespace

}  // namespace kda

extern "C" kda_status kda_verify_drafts(const int64_t* draft_tokens, const void* draft_probs, const long long* draft_strides,
                                        const void* target_probs, const long long* target_strides, const float* uniform,
                                        int64_t* tokens, int32_t* num_accepted, int N, int S, int V, unsigned flags,
                                        void* workspace, cudaStream_t stream) {
    using namespace kda;
    if (N < 1 || S < 0 || V < 1 || N > (1 << 24) || V > (1 << 30) || S > (1 << 30)) return KDA_ERR_INVALID_ARG;   // (steps of 512 in 32 bits)
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
    const bool aligned = !off(target_probs, 16) && !off(draft_probs, 16) && p.p_n % pieces == 0 && p.p_s % pieces == 0 &&
                     p.q_n % pieces == 0 && p.q_s % pieces == 0;
    // As many CTAs a sequence as fit the GPU at once (two an SM) and have 512 elements a warp (128 sequences of 131072, us
    // with 2 / 4 / 8: 22 / 27 / 37; 64 with 4 / 8: 14 / 19; 100 with 2 / 3: 21 / 23; 256 of 50257 in bf16 with 1 / 2 / 4:
    // 19 / 28 / 38).
    int ctas = 1;
    while (ctas < DR_MOST && (long long)ctas * DR_WARPS * 512 < V && 2ll * ctas * N <= 304) ctas *= 2;
    p.seg = (int)((V + (aligned ? 0 : pieces - 1) + ctas * DR_WARPS * 512 - 1) / (ctas * DR_WARPS * 512) * 512);   // with room for the shift
    // ranges a power of two apart meet in the same parts of the memory (256 x 131072 in fp32 44 us, so 41; 160 of them 37, 34)
    if (p.seg * size >= 32768u && p.seg * size % 8192u == 0) p.seg += 512;
    if (p.status && !succeeded(cudaMemsetAsync(p.status, 0, WS_CLEAR, stream))) return KDA_ERR_CUDA;
    const cudaError_t e = (flags & KDA_FLAG_FP32) != 0u   ? launch<float>(p, aligned, N, ctas, stream)
                          : (flags & KDA_FLAG_FP16) != 0u ? launch<__half>(p, aligned, N, ctas, stream)
                                                          : launch<__nv_bfloat16>(p, aligned, N, ctas, stream);
    return succeeded(e) ? KDA_OK : KDA_ERR_CUDA;
}
