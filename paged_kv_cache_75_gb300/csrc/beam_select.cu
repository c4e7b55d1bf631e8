// Selection of beam search: the K best continuations over a request's beams and
// the vocabulary (pa_beam_select).
//
// "Как работает paged attention? (детально)" 3.3 has the beams of a request share
// their blocks; which of them go on, and with which tokens, is decided here.  For the
// beams r of a request with score c_r and logits x_ri:
//     s(r, i) = c_r + ((x_ri - m_r) - log sum_j exp(x_rj - m_r)),   m_r = max_j x_rj
// and the K largest s of all (r, i) are wanted.  Within a row the order of s is the
// order of x, so one pass over the logits gives both what the sum needs and the row's
// K candidates.
//
// Rows kernel: a block holds a chunk of one row in shared memory, read once.  The K-th
// largest of its threads' maxima bounds the chunk's K-th largest element from below
// (K threads hold an element of at least it), so what passes this threshold is a short
// list that holds the chunk's K largest.  The threshold is found by bisection over
// the order-preserving integers of the maxima, one counting barrier a step.  All
// other elements go into the sum of exponentials against the chunk's maximum.
// Request kernel: the chunks' sums and candidates make each row's sum, then the K
// best of the request's rows are found the same way.
//
// Candidates of different beams are told apart beyond binary32.  A chunk's candidates
// are left out of its sum and go into the row's in full, each exponential taken to about
// 2^-30; the others' exponentials (ex2.approx, 2^-22 each, their errors unlike from
// element to element) are summed 64 at a time in binary32 and from there on in units of
// 2^-40, which no order of addition changes.  s is the sum of two floats (48 bits).
//
// 512 rows of 128256 bf16 (131 MB, 19 us at the copy rate), K = 16: rows 39 us, requests
// 14.  The rows kernel's loads alone take 27 us of that (a block's barrier, copy and wait one
// after another, five blocks an SM); then 40 instructions for eight elements' exponentials
// (maximum, unpacking, fused multiply-add, ex2, sum), 42 a group of eight that holds one
// of the list, and the list's end, some 1500 cycles a block.  Two chunks a block with the next
// one's copy ahead: 69 us (24 warps an SM instead of 40); 128 elements a thread: 43.
#include <cmath>

#include "common.cuh"
#include "launch.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxSelect = 64;
constexpr int kRowsHere = 256;  // rows of a request whose sums stay in shared memory
constexpr int kMaxVocab = 1 << 23;  // so many exponentials in units of 2^-40 fit 64 bits
constexpr int kList = 1024;  // candidates a block ranks in shared memory
constexpr float kLog2e = 1.4426950408889634f;

// A row's log-sum-exp as its two terms: added up, a large maximum would take the
// logarithm's bits with it.
struct RowSum {
    float top;           // the row's largest logit
    float log_h, log_l;  // log of the sum of exp(x - top), as the sum of two floats; log_h = +inf: the row offers nothing
    int32_t unused;
};

struct ChunkHead {
    uint64_t sum;  // of exp(x - top) over what is not in the chunk's list, in units of 2^-40
    float top;     // -inf: the chunk offers nothing
    int32_t bad;   // an allowed logit is NaN or +inf
};

struct SelectParams {
    float* scores_out;
    int32_t* rows_out;
    int32_t* tokens_out;
    const void* logits;
    const float* scores;
    const int32_t* cu_beams;
    const uint32_t* allowed;  // NULL: every token
    const uint8_t* ended;     // NULL: no row
    int32_t* status;
    RowSum* sums;              // [num_rows]
    ChunkHead* heads;   // [num_rows][chunks_per_row]
    uint64_t* keys;            // [num_rows][chunks_per_row][select]
    int64_t row_stride;
    int64_t allowed_stride;
    int32_t vocab;
    int32_t num_rows;
    int32_t num_requests;
    int32_t select;
    int32_t end_token;
    int32_t chunks_per_row;
};


// Order-preserving integer of a float (+0 and -0 alike).
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
constexpr uint32_t kNothing = 0x007fffffu;  // order_of(-inf)

__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ln 2 as 12 bits, 12 bits and the rest
constexpr double kLn2 = 0.693147180559945309417;
constexpr float kLn2a = static_cast<float>(static_cast<int>(kLn2 * 4096.0)) / 4096.f;
constexpr float kLn2b = static_cast<float>(static_cast<int>((kLn2 - kLn2a) * 16777216.0)) / 16777216.f;
constexpr float kLn2c = static_cast<float>(kLn2 - kLn2a - kLn2b);

// exp(a - b) in units of 2^-40, a <= b both finite, off by about 2^-30 of itself: the
// difference as a sum of two floats, less a whole multiple n of ln 2 (three floats of
// few bits, so that n times the first two is exact), then 1 + r + r^2/2 as a sum of two floats
// and the rest of the series, below 0.01, in one.
__device__ __forceinline__ uint64_t exp_units(float a, float b) {
    const float d = a - b;
    if (!(d > -40.f)) return 0;  // below 2^-57
    const float back = d - a;
    const float dl = (a - (d - back)) - (b + back);  // d + dl = a - b exactly
    const float n = rintf(d * kLog2e);
    const float h = fmaf(-n, kLn2a, d);  // exact: d and n kLn2a nearly cancel
    const float t = -n * kLn2b;          // exact
    const float rh = h + t;
    const float bb = rh - h;
    const float rl = ((h - (rh - bb)) + (t - bb)) + fmaf(-n, kLn2c, dl);
    const float r = rh + rl;
    // r^3/6 + r^4/24 + ..., |r| <= 0.35
    float q = 1.f / 40320.f;
    q = fmaf(q, r, 1.f / 5040.f);
    q = fmaf(q, r, 1.f / 720.f);
    q = fmaf(q, r, 1.f / 120.f);
    q = fmaf(q, r, 1.f / 24.f);
    q = fmaf(q, r, 1.f / 6.f);
    q = q * r * r * r;
    // 1 + rh + rh^2/2 + (rl + rh rl + q)
    const float s = 0.5f * rh * rh, sl = fmaf(0.5f * rh, rh, -s);
    const float u = 1.f + rh, ul = rh - (u - 1.f);
    const float v = u + s, vb = v - u;
    const float vl = (u - (v - vb)) + (s - vb);
    const float lo = vl + ul + sl + fmaf(rh, rl, rl) + q;
    const float up = exp2f(n + 40.f);  // n + 40 in [-18, 40]: exact
    return static_cast<uint64_t>(static_cast<int64_t>(__float2ll_rn(v * up)) + static_cast<int64_t>(__float2ll_rn(lo * up)));
}

// of two pairs of 16-bit floats, NaN where either is
template <int DT>
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    if constexpr (DT == PA_BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

template <int DT, typename T>
__device__ __forceinline__ float value_at(T x) {
    if constexpr (DT == PA_F32) return __uint_as_float(x);
    else return kv_pair<DT>(x).x;
}

template <int DT>
struct Logits {  // 16-bit types, two to a word
    using type = uint16_t;
    static constexpr int kVec = 8, kPerWord = 2;
    static constexpr type kNone = DT == PA_BF16 ? 0xff80u : 0xfc00u;  // -inf
};
template <>
struct Logits<PA_F32> {
    using type = uint32_t;
    static constexpr int kVec = 4, kPerWord = 1;
    static constexpr type kNone = 0xff800000u;
};

// sum over the block; all threads get it
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* scratch) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = scratch[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) v += scratch[w];
    return v;
}

// A threshold that at least `want` of the block's keys reach, found in a few steps: it
// stops once no more than 1.5 want do, or at the largest such threshold.  Where no more
// than `want` keys are above kNothing, what all of those reach.  top: the block's largest
// key (> kNothing).  DROP: low bits that say nothing (a 16-bit type's values: a step a
// value, not 2^16 of them).  scratch: a word a warp.
template <int DROP>
__device__ __forceinline__ uint32_t threshold(uint32_t key, uint32_t top, int want, uint32_t* scratch) {
    if (__syncthreads_count(key > kNothing) <= want) return kNothing + 1;
    // (the keys lie close together in the range of all floats: start from the least)
    uint32_t lo = __reduce_min_sync(0xffffffffu, key > kNothing ? key : top) >> DROP, hi = top >> DROP;
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = lo;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) lo = min(lo, scratch[w]);
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        const int n = __syncthreads_count(key >> DROP >= mid);
        if (n >= want) {
            lo = mid;
            if (n <= want + want / 2) break;
        } else {
            hi = mid - 1;
        }
    }
    return lo << DROP;
}

// One chunk's list and sum (see beam_rows_kernel): element first + i is mem[i].
template <int DT, int EPT, bool VEC>
__device__ __forceinline__ void rows_chunk(const SelectParams& p, typename Logits<DT>::type* mem,
                                           const typename Logits<DT>::type* chunk_mem, int skew, int first, int here,
                                           int64_t row, ChunkHead* head, uint64_t* keys, uint64_t* list, int& list_n,
                                           uint64_t* scratch64, float* scratch, uint32_t* scratch32) {
    using L = Logits<DT>;
    constexpr int kChunk = kThreads * EPT, kGroups = EPT / 8;
    const int t = threadIdx.x, lane = t & 31;
    // element of group g that comes first, and how far the others are apart
    auto place = [&](int g, int i, int t) -> int {  // of thread t
        if constexpr (VEC) {
            constexpr int kVecs = 8 / L::kVec;  // vectors of a group
            return ((g * kVecs + i / L::kVec) * kThreads + t) * L::kVec + i % L::kVec;
        } else {
            constexpr int kWords = 8 / L::kPerWord;
            return ((g * kWords + i / L::kPerWord) * kThreads + t) * L::kPerWord + i % L::kPerWord;
        }
    };
    // what the row does not have or may not take: -inf
    if (here < kChunk || p.allowed != nullptr) {
        const uint32_t* bits = p.allowed == nullptr ? nullptr : p.allowed + row * p.allowed_stride;
#pragma unroll 1
        for (int g = 0; g < kGroups; ++g) {
#pragma unroll
            for (int w = 0; w < 8; w += VEC ? L::kVec : L::kPerWord) {
                // (these neighbours' bits lie in one word)
                const int i0 = place(g, w, t);
                uint32_t on = 0;
                if (i0 < here) on = bits != nullptr ? __ldg(bits + ((first + i0) >> 5)) >> ((first + i0) & 31) : ~0u;
#pragma unroll
                for (int i = 0; i < (VEC ? L::kVec : L::kPerWord); ++i)
                    if (i0 + i >= here || !(on >> i & 1u)) mem[i0 + i] = L::kNone;
            }
        }
        if constexpr (!VEC) __syncthreads();  // (a pair's words hold other threads' elements too)
    }
    // group g's elements: two to a word (16-bit types), or one
    constexpr int kGroupWords = 8 / L::kPerWord;
    auto words = [&](int g, uint32_t (&w)[kGroupWords]) {
        if constexpr (VEC) {
#pragma unroll
            for (int v = 0; v < kGroupWords / 4; ++v) {
                const uint4 x = *reinterpret_cast<const uint4*>(mem + place(g, v * L::kVec, t));
                w[4 * v] = x.x;
                w[4 * v + 1] = x.y;
                w[4 * v + 2] = x.z;
                w[4 * v + 3] = x.w;
            }
        } else if constexpr (L::kPerWord == 2) {
            const uint32_t* m = reinterpret_cast<const uint32_t*>(chunk_mem + (skew & ~1));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int at = place(g, 2 * k, t) / 2;
                w[k] = skew & 1 ? __funnelshift_r(m[at], m[at + 1], 16) : m[at];
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = mem[place(g, k, t)];
        }
    };
    auto element = [&](const uint32_t (&w)[kGroupWords], int i) -> float {
        if constexpr (L::kPerWord == 2) {
            const float2 f = kv_pair<DT>(w[i / 2]);
            return i & 1 ? f.y : f.x;
        } else {
            return __uint_as_float(w[i]);
        }
    };
    auto largest = [&](const uint32_t (&w)[kGroupWords]) -> float {
        if constexpr (L::kPerWord == 2) {
            const float2 f = kv_pair<DT>(max2_nan<DT>(max2_nan<DT>(w[0], w[1]), max2_nan<DT>(w[2], w[3])));
            return max_nan(f.x, f.y);
        } else {
            float m = __uint_as_float(w[0]);
#pragma unroll
            for (int i = 1; i < 8; ++i) m = max_nan(m, __uint_as_float(w[i]));
            return m;
        }
    };
    auto key_of = [&](int g, const uint32_t (&w)[kGroupWords], int i) -> uint64_t {
        return (static_cast<uint64_t>(order_of(element(w, i))) << 32) | static_cast<uint32_t>(~(first + place(g, i, t)));
    };
    // ---- maxima: the thread's, the block's ----
    float gmax[kGroups], mine = -INFINITY;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        uint32_t w[kGroupWords];
        words(g, w);
        gmax[g] = largest(w);
        mine = max_nan(mine, gmax[g]);
    }
    float top = mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((t & 31) == 0) scratch[t >> 5] = top;
    __syncthreads();
    top = scratch[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) top = max_nan(top, scratch[w]);
    if (!(top < INFINITY) || top == -INFINITY) {
        if (t == 0) *head = {0, -INFINITY, !(top < INFINITY) ? 1 : 0};
        if (t < p.select) keys[t] = 0;
        return;
    }
    const uint32_t cut = threshold<DT == PA_BF16 ? 16 : DT == PA_F16 ? 13 : 0>(order_of(mine), order_of(top), p.select, scratch32);
    const float cut_v = value_of(cut);
    // ---- the list of what reaches the threshold; the sum of the rest ----
    // exp(x - top) as 2^(x L - h), L = log2 e and h = top L rounded down: one fused
    // multiply-add, whose product is exact, so a large common part of the logits takes
    // nothing; the sum is 2^(top L - h) too large, which is put right below.  (Logits so
    // large that their differences are zero or past any exponential: zero, what equals
    // top being in the list.)
    const bool huge = !(fabsf(top) < 1e30f);
    const float mult = huge ? 1e-30f : kLog2e, h = huge ? 1e9f : __fmul_rd(top, kLog2e);
    auto exp_of = [&](float x) -> float { return exp2_approx(fmaf(x, mult, -h)); };
    float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        uint32_t w[kGroupWords];
        words(g, w);
        float s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = exp_of(element(w, 2 * i)) + exp_of(element(w, 2 * i + 1));
        const bool mixed = gmax[g] >= cut_v;
        sum0 += mixed ? 0.f : (s[0] + s[1]) + (s[2] + s[3]);
        // groups that hold one of the list (a few in a hundred): eight lanes take the
        // eight elements of one
        for (uint32_t who = __ballot_sync(0xffffffffu, mixed); who != 0; who &= who - 1) {
            const int at = place(g, lane & 7, (t & ~31) + __ffs(who) - 1);
            const float x = lane < 8 ? value_at<DT>(mem[at]) : -INFINITY;
            if (x >= cut_v) {
                const int n = atomicAdd(&list_n, 1);
                if (n < kList) list[n] = (static_cast<uint64_t>(order_of(x)) << 32) | static_cast<uint32_t>(~(first + at));
            } else {
                sum1 += exp_of(x);
            }
        }
    }
    // 1 - 2^-(top L - h), to a few times its own 2^-24
    const float u = huge ? 0.f : fmaf(top, kLog2e, -h) * static_cast<float>(kLn2);
    const float over = u * fmaf(u, fmaf(u, fmaf(u, fmaf(u, 1.f / 120.f, -1.f / 24.f), 1.f / 6.f), -0.5f), 1.f);
    auto units_of = [&](float x) -> uint64_t {
        const float y = x * 1099511627776.f;
        return static_cast<uint64_t>(__float2ll_rn(y) - __float2ll_rn(y * over));
    };
    uint64_t units = units_of(sum0 + sum1);
    __syncthreads();
    const int n = list_n;
    if (n <= kList) {
        // by rank: how many of the list are larger (keys differ: each has its token)
        for (int i = t; i < n; i += kThreads) {
            const uint64_t k = list[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += list[j] > k;
            if (rank < p.select) keys[rank] = k;
            else units += exp_units(value_of(static_cast<uint32_t>(k >> 32)), top);
        }
        if (t >= n && t < p.select) keys[t] = 0;
    } else {
        // more than the list holds (many equal logits, or few threads with any): one
        // candidate a round, the largest below the last one
        uint64_t last = ~0ull;
        for (int r = 0; r < p.select; ++r) {
            uint64_t best = 0;
#pragma unroll 1
            for (int g = 0; g < kGroups; ++g) {
                uint32_t w[kGroupWords];
                words(g, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint64_t k = key_of(g, w, i);
                    if (element(w, i) > -INFINITY && k < last && k > best) best = k;
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const uint64_t y = __shfl_xor_sync(0xffffffffu, best, o);
                if (y > best) best = y;
            }
            __syncthreads();
            if ((t & 31) == 0) scratch64[t >> 5] = best;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w)
                if (scratch64[w] > best) best = scratch64[w];
            last = best;  // (0 once nothing is left: the rounds that follow find nothing)
            if (t == 0) keys[r] = best;
        }
        // the sum again, over all but the candidates
        units = 0;
#pragma unroll 1
        for (int g = 0; g < kGroups; ++g) {
            uint32_t w[kGroupWords];
            words(g, w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (element(w, i) > -INFINITY && key_of(g, w, i) < last)
                    units += units_of(huge ? (element(w, i) == top ? 1.f : 0.f) : exp_of(element(w, i)));
        }
    }
    units = block_sum(units, scratch64);
    if (t == 0) *head = {units, top, 0};
}

// EPT elements a thread, in groups of eight.  VEC: every row is 16-byte aligned and a group
// is whole vectors of shared memory; otherwise it is four words' pairs of 16-bit elements
// (eight floats), which lie in shared memory as they lie in memory, up to 14 bytes behind
// a vector's start.  Which element goes to which thread does not depend on a row's
// address, so equal rows get equal sums.
template <int DT, int EPT, bool VEC>
__global__ void __launch_bounds__(kThreads)
beam_rows_kernel(const SelectParams p) {
    using L = Logits<DT>;
    using T = typename L::type;
    constexpr int kChunk = kThreads * EPT;
    extern __shared__ __align__(16) uint8_t dynamic[];  // [kChunk + kVec] T
    __shared__ uint64_t list[kList];
    __shared__ uint64_t scratch64[kThreads / 32];
    __shared__ float scratch[kThreads / 32];
    __shared__ uint32_t scratch32[kThreads / 32];
    __shared__ uint64_t full;
    __shared__ int list_n, abort_flag;

    const int t = threadIdx.x;
    const int row = blockIdx.x / p.chunks_per_row, first = (blockIdx.x - row * p.chunks_per_row) * kChunk;
    const int here = min(kChunk, p.vocab - first);
    if (t == 0) {
        mbar_init(smem_addr(&full), 1);
        list_n = 0;
        abort_flag = 0;
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    ChunkHead* head = p.heads + blockIdx.x;
    uint64_t* keys = p.keys + static_cast<int64_t>(blockIdx.x) * p.select;
    // a beam that ended, or that a request does not have yet, is not read
    const bool live = !(p.ended != nullptr && p.ended[row] != 0) && p.scores[row] > -INFINITY && p.scores[row] < INFINITY;
    if (!live) {
        if (t == 0) *head = {0, -INFINITY, 0};
        if (t < p.select) keys[t] = 0;
        return;
    }
    // the chunk into shared memory, at its own offset from a vector's start: whole
    // vectors by one bulk copy, the up to 7 elements before and behind them by element
    const T* src = static_cast<const T*>(p.logits) + row * p.row_stride + first;
    const int skew = VEC ? 0 : static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15u) / sizeof(T));
    T* mem = reinterpret_cast<T*>(dynamic) + skew;  // element first + i is mem[i]
    const int lead = skew == 0 ? 0 : min(here, L::kVec - skew), vecs = (here - lead) / L::kVec;
    if (t == 0) {
        if (vecs > 0) {
            mbar_expect_tx(smem_addr(&full), vecs * 16);
            bulk_g2s_hint(smem_addr(mem + lead), src + lead, vecs * 16, smem_addr(&full), policy_evict_first());
        } else {
            mbar_arrive(smem_addr(&full));
        }
    }
    if (t < lead) mem[t] = src[t];
    if (lead + vecs * L::kVec + t < here) mem[lead + vecs * L::kVec + t] = src[lead + vecs * L::kVec + t];
    __syncthreads();  // (the barrier's initialisation, the single elements)
    // (one outcome for the block: a wait that ran out ends it)
    if (__syncthreads_or(!mbar_wait(smem_addr(&full), 0u, p.status, &abort_flag))) return;
    rows_chunk<DT, EPT, VEC>(p, mem, reinterpret_cast<T*>(dynamic), skew, first, here, row, head, keys, list, list_n, scratch64,
                             scratch, scratch32);
}

// A number as the sum of two floats, hi the sum rounded: 48 bits.  Below binary32's range
// it is hi alone.
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = a + b, bb = s - a;
    return {s, s > -INFINITY ? (a - (s - bb)) + (b - bb) : 0.f};
}
__device__ __forceinline__ Two two_add(Two a, Two b) {
    Two s = two_sum(a.hi, b.hi);
    if (!(s.hi > -INFINITY)) return s;
    s.lo += a.lo + b.lo;
    return two_sum(s.hi, s.lo);
}

// log(units 2^-40), units >= 2^40 or a little less, to about 2^-29: the power of two apart,
// then log m = y + (m exp(-y) - 1) for y the binary32 logarithm
__device__ __forceinline__ Two log_units(uint64_t units) {
    const int k = 23 - __clzll(static_cast<int64_t>(units));  // units = m 2^k, m in [2^40, 2^41)
    const uint64_t m = k >= 0 ? units >> k : units << -k;
    const float y = __logf(static_cast<float>(m) * 9.094947017729282e-13f);  // (2^-40)
    const uint64_t e = exp_units(-y, 0.f);
    const int64_t more = static_cast<int64_t>((__umul64hi(m, e) << 24) | (m * e >> 40)) - (1ll << 40);
    const float f = static_cast<float>(k);
    // k ln 2 in the same three terms, the first two exact
    const Two a = two_sum(f * kLn2a, f * kLn2b);
    return two_add(two_add(a, {f * kLn2c, 0.f}), two_sum(y, static_cast<float>(more) * 9.094947017729282e-13f));
}

struct Candidate {
    Two s;
    uint64_t key;  // the logit's order, then the token's complement
    int32_t row;
};
// c stands before d: by score, then row; of one row by logit (a large maximum can take
// the difference from their scores), then token
__device__ __forceinline__ bool before(const Candidate& c, const Candidate& d) {
    if (c.s.hi != d.s.hi) return c.s.hi > d.s.hi;
    if (c.s.lo != d.s.lo) return c.s.lo > d.s.lo;
    if (c.row != d.row) return c.row < d.row;
    return c.key > d.key;
}

// One block a request.
__global__ void __launch_bounds__(kThreads)
beam_requests_kernel(const SelectParams p) {
    __shared__ Candidate list[kList];
    __shared__ Candidate warp_best[kThreads / 32];
    __shared__ RowSum row_sums[kRowsHere];
    __shared__ uint32_t scratch[kThreads / 32];
    __shared__ int list_n;
    pdl_wait();
    pdl_trigger();
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int K = p.select, S = p.chunks_per_row;
    const int64_t out0 = static_cast<int64_t>(blockIdx.x) * K;
    int r0 = p.cu_beams[blockIdx.x], r1 = p.cu_beams[blockIdx.x + 1];
    if (r0 < 0 || r1 < r0 || r1 > p.num_rows) {
        if (t == 0) report(p.status, PA_ERR_INVALID_ARG);
        r0 = r1 = 0;
    }
    if (t == 0) list_n = 0;
    RowSum* sums = r1 - r0 <= kRowsHere ? row_sums : p.sums + r0;
    // a key's candidate: score + ((x - top) - log)
    auto scored = [&](int row, float score, const RowSum& sum, uint64_t key) -> Candidate {
        const float x = value_of(static_cast<uint32_t>(key >> 32));
        return {two_add(two_add(two_sum(x, -sum.top), {-sum.log_h, -sum.log_l}), {score, 0.f}), key, row};
    };
    // (the score's float keeps the scores' order, so it serves as the threshold's key)
    auto order = [](const Candidate& c) -> uint32_t { return order_of(fmaxf(c.s.hi, -3.4028234e38f)); };
    // use(candidate) for all that this thread looks at.  A warp takes a row, or, of few
    // rows, several warps do.
    const int per_row = S * K, sharers = max(1, min(kThreads / 32, kThreads / 32 / max(r1 - r0, 1)));
    auto candidates = [&](auto use) {
        for (int row = r0 + warp / sharers; row < r1 && warp / sharers < kThreads / 32 / sharers;
             row += kThreads / 32 / sharers) {
            const float score = p.scores[row];
            if (!(score > -INFINITY && score < INFINITY)) continue;
            const int first = (warp % sharers) * 32 + lane;
            if (p.ended != nullptr && p.ended[row] != 0) {
                if (first == 0) use(Candidate{{score, 0.f}, static_cast<uint32_t>(~p.end_token), row});
                continue;
            }
            const RowSum sum = sums[row - r0];
            if (sum.log_h == INFINITY) continue;
            const uint64_t* keys = p.keys + static_cast<int64_t>(row) * per_row;
            for (int i = first; i < per_row; i += 32 * sharers)
                if (keys[i] != 0) use(scored(row, score, sum, keys[i]));
        }
    };
    // ---- each row's log-sum-exp, by a warp ----
    for (int row = r0 + warp; row < r1; row += kThreads / 32) {
        const float score = p.scores[row];
        if (!(score < INFINITY) && lane == 0) report(p.status, PA_ERR_INVALID_ARG);
        const ChunkHead* heads = p.heads + static_cast<int64_t>(row) * S;
        const uint64_t* keys = p.keys + static_cast<int64_t>(row) * per_row;
        float top = -INFINITY;
        bool bad = false;
        for (int c = lane; c < S; c += 32) {
            top = fmaxf(top, heads[c].top);
            bad |= heads[c].bad != 0;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        bad = __any_sync(0xffffffffu, bad);
        if (bad && lane == 0) report(p.status, PA_ERR_INVALID_ARG);
        RowSum sum{top, INFINITY, 0.f, 0};
        if (!bad && top > -INFINITY) {
            uint64_t units = 0;
#pragma unroll 4
            for (int i = lane; i < per_row; i += 32) {
                const uint64_t k = keys[i];
                if (k != 0) units += exp_units(value_of(static_cast<uint32_t>(k >> 32)), top);
            }
            // (a chunk's units count against its own maximum)
            for (int c = lane; c < S; c += 32) {
                const uint64_t u = heads[c].sum, e = u != 0 ? exp_units(heads[c].top, top) : 0;
                units += (__umul64hi(u, e) << 24) | (u * e >> 40);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) units += __shfl_xor_sync(0xffffffffu, units, o);
            const Two l = log_units(units);
            sum.log_h = l.hi;
            sum.log_l = l.lo;
        }
        if (lane == 0) sums[row - r0] = sum;
    }
    __syncthreads();
    // ---- the K best of all candidates ----
    uint32_t mine = kNothing;
    candidates([&](const Candidate& c) { mine = max(mine, order(c)); });
    uint32_t top = __reduce_max_sync(0xffffffffu, mine);
    if (lane == 0) scratch[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) top = max(top, scratch[w]);
    const uint32_t cut = top == kNothing ? kNothing + 1 : threshold<0>(mine, top, K, scratch);
    if (__any_sync(0xffffffffu, mine >= cut)) {
        candidates([&](const Candidate& c) {
            if (order(c) < cut) return;
            const int n = atomicAdd(&list_n, 1);
            if (n < kList) list[n] = c;
        });
    }
    __syncthreads();
    const int n = list_n;
    auto put = [&](int rank, const Candidate& c) {
        p.scores_out[out0 + rank] = c.s.hi;
        p.rows_out[out0 + rank] = c.row;
        p.tokens_out[out0 + rank] = c.row < 0 ? -1 : static_cast<int32_t>(~static_cast<uint32_t>(c.key));
    };
    const Candidate none{{-INFINITY, 0.f}, 0, -1};
    if (n <= kList) {
        for (int i = warp; i < n; i += kThreads / 32) {
            const Candidate c = list[i];
            int rank = 0;
            for (int j = 0; j < n; j += 32)
                rank += __popc(__ballot_sync(0xffffffffu, j + lane < n && before(list[min(j + lane, n - 1)], c)));
            if (rank < K && lane == 0) put(rank, c);
        }
        if (t >= n && t < K) put(t, none);
        return;
    }
    // more than the list holds: one a round, the first behind the last one
    Candidate last{{INFINITY, 0.f}, 0, -1};
    for (int r = 0; r < K; ++r) {
        Candidate best = none;
        candidates([&](const Candidate& c) {
            if (before(last, c) && (best.row < 0 || before(c, best))) best = c;
        });
        auto join = [&](const Candidate& c) {
            if (c.row >= 0 && (best.row < 0 || before(c, best))) best = c;
        };
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const Candidate c{{__shfl_xor_sync(0xffffffffu, best.s.hi, o), __shfl_xor_sync(0xffffffffu, best.s.lo, o)},
                              __shfl_xor_sync(0xffffffffu, best.key, o), __shfl_xor_sync(0xffffffffu, best.row, o)};
            join(c);
        }
        __syncthreads();
        if (lane == 0) warp_best[warp] = best;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) join(warp_best[w]);
        // (more candidates than the list holds are more than K: best is one)
        if (t == 0) put(r, best);
        last = best;
    }
}

// Elements a thread holds: more of them share a chunk's threshold and list (some 2700
// instructions), fewer keep more blocks on an SM (512 rows of 128256 bf16: 64 elements
// 40.5 us, 128 elements 43.1) and reach every SM with a small batch.
int chunk_elems(int64_t rows, int vocab, int dtype, int sms) {
    int ept = dtype == PA_F32 ? 32 : 64;
    while (ept > 8 && rows * ((vocab + kThreads * ept - 1) / (kThreads * ept)) < 2ll * sms) ept /= 2;
    return ept;
}
int chunks_of(int vocab, int ept) { return (vocab + kThreads * ept - 1) / (kThreads * ept); }

template <int DT, int EPT, bool VEC>
cudaError_t launch_rows_of(const SelectParams& p, int items, cudaStream_t s) {
    const int smem = (kThreads * EPT + Logits<DT>::kVec) * static_cast<int>(sizeof(typename Logits<DT>::type));
    static LaunchCache cache;
    if (blocks_per_sm(beam_rows_kernel<DT, EPT, VEC>, kThreads, smem, cache) <= 0) return cudaErrorUnknown;
    return launch_pdl(beam_rows_kernel<DT, EPT, VEC>, items, kThreads, smem, s, p);
}
template <int DT, bool VEC>
cudaError_t launch_rows(const SelectParams& p, int ept, int items, cudaStream_t s) {
    if constexpr (DT != PA_F32)
        if (ept == 64) return launch_rows_of<DT, 64, VEC>(p, items, s);
    if (ept == 32) return launch_rows_of<DT, 32, VEC>(p, items, s);
    if (ept == 16) return launch_rows_of<DT, 16, VEC>(p, items, s);
    return launch_rows_of<DT, 8, VEC>(p, items, s);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_beam_select_workspace_size(int32_t num_rows, int32_t vocab, int32_t num_select) {
    if (num_rows <= 0 || vocab <= 0 || num_select <= 0 || num_select > kMaxSelect) return 0;
    // (for the shortest chunks, which any device may take)
    const size_t chunks = static_cast<size_t>(num_rows) * chunks_of(vocab, 8);
    return static_cast<size_t>(num_rows) * sizeof(RowSum) + chunks * (sizeof(ChunkHead) + 8 * static_cast<size_t>(num_select));
}

extern "C" pa_status pa_beam_select(float* scores_out, int32_t* rows_out, int32_t* tokens_out, const void* logits,
                                    pa_dtype dtype, int64_t row_stride, int32_t vocab, int32_t num_rows,
                                    const float* scores, const int32_t* cu_beams, int32_t num_requests,
                                    const uint32_t* allowed, int64_t allowed_stride, const uint8_t* ended,
                                    int32_t end_token, int32_t num_select, void* workspace, size_t workspace_bytes,
                                    int32_t* dev_status, pa_stream_t stream) {
    if (dtype != PA_F16 && dtype != PA_BF16 && dtype != PA_F32) return PA_ERR_UNSUPPORTED;
    if (num_requests < 0 || num_rows < 0 || vocab <= 0 || num_select <= 0 || row_stride < vocab) return PA_ERR_INVALID_ARG;
    if (num_select > kMaxSelect || vocab > kMaxVocab) return PA_ERR_UNSUPPORTED;
    if (num_requests == 0) return PA_OK;
    if (scores_out == nullptr || rows_out == nullptr || tokens_out == nullptr || cu_beams == nullptr)
        return PA_ERR_INVALID_ARG;
    if (num_rows > 0 && (logits == nullptr || scores == nullptr)) return PA_ERR_INVALID_ARG;
    const uintptr_t bytes = dtype == PA_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(logits) & (bytes - 1)) return PA_ERR_INVALID_ARG;
    if (allowed != nullptr && allowed_stride < (static_cast<int64_t>(vocab) + 31) / 32) return PA_ERR_INVALID_ARG;
    if (ended != nullptr && (end_token < 0 || end_token >= vocab)) return PA_ERR_INVALID_ARG;
    const size_t need = pa_beam_select_workspace_size(num_rows, vocab, num_select);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 15u)))
        return PA_ERR_INVALID_ARG;
    const int sms = device_sm_count();
    if (sms <= 0) return PA_ERR_CUDA;

    SelectParams p{};
    p.scores_out = scores_out;
    p.rows_out = rows_out;
    p.tokens_out = tokens_out;
    p.logits = logits;
    p.scores = scores;
    p.cu_beams = cu_beams;
    p.allowed = allowed;
    p.ended = ended;
    p.status = dev_status;
    p.row_stride = row_stride;
    p.allowed_stride = allowed_stride;
    p.vocab = vocab;
    p.num_rows = num_rows;
    p.num_requests = num_requests;
    p.select = num_select;
    p.end_token = end_token;
    const int ept = chunk_elems(num_rows, vocab, dtype, sms);
    p.chunks_per_row = chunks_of(vocab, ept);
    p.sums = static_cast<RowSum*>(workspace);
    p.heads = reinterpret_cast<ChunkHead*>(p.sums + num_rows);
    p.keys = reinterpret_cast<uint64_t*>(p.heads + static_cast<int64_t>(num_rows) * p.chunks_per_row);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (num_rows > 0) {
        const int64_t grid = static_cast<int64_t>(num_rows) * p.chunks_per_row;
        if (grid > INT32_MAX / 2) return PA_ERR_UNSUPPORTED;
        const bool vec = (reinterpret_cast<uintptr_t>(logits) & 15u) == 0 && (row_stride * bytes) % 16 == 0;
        const int g = static_cast<int>(grid);
        cudaError_t e;
        if (dtype == PA_F32) e = vec ? launch_rows<PA_F32, true>(p, ept, g, s) : launch_rows<PA_F32, false>(p, ept, g, s);
        else if (dtype == PA_F16) e = vec ? launch_rows<PA_F16, true>(p, ept, g, s) : launch_rows<PA_F16, false>(p, ept, g, s);
        else e = vec ? launch_rows<PA_BF16, true>(p, ept, g, s) : launch_rows<PA_BF16, false>(p, ept, g, s);
        if (e != cudaSuccess) return PA_ERR_CUDA;
    }
    return launch_pdl(beam_requests_kernel, num_requests, kThreads, 0, s, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
