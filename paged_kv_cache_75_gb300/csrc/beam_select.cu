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
    uint8_t* chunks;  // [num_rows][chunks_per_row] of chunk_bytes: header, then `select` keys
    RowSum* sums;  // [num_rows]
    int64_t row_stride;
    int64_t allowed_stride;
    int32_t vocab;
    int32_t num_rows;
    int32_t num_requests;
    int32_t select;
    int32_t end_token;
    int32_t chunks_per_row;
    int32_t chunk_bytes;
};

struct ChunkHead {
    uint64_t sum;  // of exp(x - top) over what is not in the chunk's list, in units of 2^-40
    float top;     // -inf: the chunk offers nothing
    int32_t bad;   // an allowed logit is NaN or +inf
};
static_assert(sizeof(ChunkHead) == 16, "the keys follow at 16 bytes");
constexpr double kUnit = 1.0 / (1ull << 40);

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

// pairs of floats, one instruction for both
__device__ __forceinline__ float2 f2_op(uint64_t r) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(r));
    return f;
}
__device__ __forceinline__ uint64_t f2_of(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 f2_add(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(f2_of(a.x, a.y)), "l"(f2_of(b.x, b.y)));
    return f2_op(d);
}
__device__ __forceinline__ float2 f2_add(float2 a, float b) { return f2_add(a, make_float2(b, b)); }
__device__ __forceinline__ float2 f2_mul(float2 a, float b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(f2_of(a.x, a.y)), "l"(f2_of(b, b)));
    return f2_op(d);
}

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
    // ln 2 = c0 + c1 + c2: 12 bits, 12 bits, the rest
    constexpr double kLn2 = 0.693147180559945309417;
    constexpr float c0 = static_cast<float>(static_cast<int>(kLn2 * 4096.0)) / 4096.f;
    constexpr float c1 = static_cast<float>(static_cast<int>((kLn2 - c0) * 16777216.0)) / 16777216.f;
    constexpr float c2 = static_cast<float>(kLn2 - c0 - c1);
    const float h = fmaf(-n, c0, d);  // exact: d and n c0 nearly cancel
    const float t = -n * c1;          // exact
    const float rh = h + t;
    const float bb = rh - h;
    const float rl = ((h - (rh - bb)) + (t - bb)) + fmaf(-n, c2, dl);
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
// key (> kNothing).  scratch: a word a warp.
__device__ __forceinline__ uint32_t threshold(uint32_t key, uint32_t top, int want, uint32_t* scratch) {
    if (__syncthreads_count(key > kNothing) <= want) return kNothing + 1;
    // (the keys lie close together in the range of all floats: start from the least)
    uint32_t lo = __reduce_min_sync(0xffffffffu, key > kNothing ? key : top), hi = top;
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = lo;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) lo = min(lo, scratch[w]);
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        const int n = __syncthreads_count(key >= mid);
        if (n >= want) {
            lo = mid;
            if (n <= want + want / 2) break;
        } else {
            hi = mid - 1;
        }
    }
    return lo;
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
    constexpr int kChunk = kThreads * EPT, kGroups = EPT / 8;
    __shared__ __align__(16) T chunk_mem[kChunk + L::kVec];
    __shared__ uint64_t list[kList];
    __shared__ uint64_t scratch64[kThreads / 32];
    __shared__ float scratch[kThreads / 32];
    __shared__ uint32_t scratch32[kThreads / 32];
    __shared__ int list_n;

    const int t = threadIdx.x;
    const int row = blockIdx.x / p.chunks_per_row, chunk = blockIdx.x - row * p.chunks_per_row;
    const int first = chunk * kChunk, here = min(kChunk, p.vocab - first);
    pdl_wait();
    pdl_trigger();
    uint8_t* base = p.chunks + static_cast<int64_t>(blockIdx.x) * p.chunk_bytes;
    ChunkHead* head = reinterpret_cast<ChunkHead*>(base);
    uint64_t* keys = reinterpret_cast<uint64_t*>(base + sizeof(ChunkHead));
    // a beam that ended, or that a request does not have yet, is not read
    const bool live = !(p.ended != nullptr && p.ended[row] != 0) && p.scores[row] > -INFINITY && p.scores[row] < INFINITY;
    if (!live) {
        if (t == 0) *head = {0, -INFINITY, 0};
        if (t < p.select) keys[t] = 0;
        return;
    }
    // ---- the chunk into shared memory, at its own offset from a vector's start ----
    const T* src = static_cast<const T*>(p.logits) + row * p.row_stride + first;
    const int skew = VEC ? 0 : static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15u) / sizeof(T));
    T* mem = chunk_mem + skew;  // element first + i is mem[i]
    {
        // whole vectors asynchronously, what is left at the two ends by element
        const int lead = skew == 0 ? 0 : min(here, L::kVec - skew), vecs = (here - lead) / L::kVec;
        for (int v = t; v < vecs; v += kThreads) {
            const int at = lead + v * L::kVec;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(mem + at)),
                         "l"(reinterpret_cast<uint64_t>(src + at))
                         : "memory");
        }
        if (t < lead) mem[t] = src[t];
        const int rest = lead + vecs * L::kVec;
        if (rest + t < here) mem[rest + t] = src[rest + t];
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
    }
    // element of group g that comes first, and how far the others are apart
    auto place = [&](int g, int i) -> int {
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
                const int i0 = place(g, w);
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
                const uint4 x = *reinterpret_cast<const uint4*>(mem + place(g, v * L::kVec));
                w[4 * v] = x.x;
                w[4 * v + 1] = x.y;
                w[4 * v + 2] = x.z;
                w[4 * v + 3] = x.w;
            }
        } else if constexpr (L::kPerWord == 2) {
            const uint32_t* m = reinterpret_cast<const uint32_t*>(chunk_mem + (skew & ~1));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int at = place(g, 2 * k) / 2;
                w[k] = skew & 1 ? __funnelshift_r(m[at], m[at + 1], 16) : m[at];
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = mem[place(g, k)];
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
        return (static_cast<uint64_t>(order_of(element(w, i))) << 32) | static_cast<uint32_t>(~(first + place(g, i)));
    };
    // ---- maxima: the thread's, the block's ----
    float mine = -INFINITY;
#pragma unroll 4
    for (int g = 0; g < kGroups; ++g) {
        uint32_t w[kGroupWords];
        words(g, w);
        mine = max_nan(mine, largest(w));
    }
    float top = mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((t & 31) == 0) scratch[t >> 5] = top;
    if (t == 0) list_n = 0;
    __syncthreads();
    top = scratch[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) top = max_nan(top, scratch[w]);
    if (!(top < INFINITY) || top == -INFINITY) {
        if (t == 0) *head = {0, -INFINITY, !(top < INFINITY) ? 1 : 0};
        if (t < p.select) keys[t] = 0;
        return;
    }
    const uint32_t cut = threshold(order_of(mine), order_of(top), p.select, scratch32);
    const float cut_v = value_of(cut);
    // ---- the list of what reaches the threshold; the sum of the rest ----
    // exp(x - top): the difference first, which is exact or nearly so (a product with
    // log2 e first would lose what a large common part of the logits takes)
    auto exp_of = [&](float x) -> float { return exp2_approx((x - top) * kLog2e); };
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int g = 0; g < kGroups; ++g) {
        uint32_t w[kGroupWords];
        words(g, w);
        if (largest(w) >= cut_v) {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                const float x = value_at<DT>(mem[place(g, i)]);
                if (x >= cut_v) {
                    const int at = atomicAdd(&list_n, 1);
                    if (at < kList)
                        list[at] = (static_cast<uint64_t>(order_of(x)) << 32) | static_cast<uint32_t>(~(first + place(g, i)));
                } else {
                    sum.x += exp_of(x);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                float2 e = f2_mul(f2_add(make_float2(element(w, i), element(w, i + 1)), -top), kLog2e);
                e.x = exp2_approx(e.x);
                e.y = exp2_approx(e.y);
                sum = f2_add(sum, e);
            }
        }
    }
    uint64_t units = static_cast<uint64_t>(__float2ll_rn((sum.x + sum.y) * 1099511627776.f));
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
                    units += static_cast<uint64_t>(__float2ll_rn(exp_of(element(w, i)) * 1099511627776.f));
        }
    }
    units = block_sum(units, scratch64);
    if (t == 0) *head = {units, top, 0};
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
    auto head_of = [&](int row, int c) -> const uint8_t* {
        return p.chunks + (static_cast<int64_t>(row) * S + c) * p.chunk_bytes;
    };
    if (t == 0) list_n = 0;
    // ---- each row's log-sum-exp: a warp takes a row, then a thread its logarithm ----
    RowSum* sums = r1 - r0 <= kRowsHere ? row_sums : p.sums + r0;
    for (int row = r0 + warp; row < r1; row += kThreads / 32) {
        const float score = p.scores[row];
        if (!(score < INFINITY) && lane == 0) report(p.status, PA_ERR_INVALID_ARG);
        float top = -INFINITY;
        bool bad = false;
        for (int c = lane; c < S; c += 32) {
            const ChunkHead h = *reinterpret_cast<const ChunkHead*>(head_of(row, c));
            top = fmaxf(top, h.top);
            bad |= h.bad != 0;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        bad = __any_sync(0xffffffffu, bad);
        if (bad && lane == 0) report(p.status, PA_ERR_INVALID_ARG);
        uint64_t units = 0;
        if (!bad && top > -INFINITY) {
            for (int i = lane; i < S * K; i += 32) {
                const int c = i / K;
                const uint64_t k = reinterpret_cast<const uint64_t*>(head_of(row, c) + sizeof(ChunkHead))[i - c * K];
                if (k != 0) units += exp_units(value_of(static_cast<uint32_t>(k >> 32)), top);
            }
            // (a chunk's units count against its own maximum)
            for (int c = lane; c < S; c += 32) {
                const ChunkHead h = *reinterpret_cast<const ChunkHead*>(head_of(row, c));
                const uint64_t e = h.sum != 0 ? exp_units(h.top, top) : 0;
                units += (__umul64hi(h.sum, e) << 24) | (h.sum * e >> 40);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) units += __shfl_xor_sync(0xffffffffu, units, o);
        }
        if (lane == 0) {
            // (the units wait where the logarithm goes)
            sums[row - r0].top = top;
            sums[row - r0].log_h = __uint_as_float(static_cast<uint32_t>(units));
            sums[row - r0].log_l = __uint_as_float(static_cast<uint32_t>(units >> 32));
        }
    }
    __syncthreads();
    for (int r = t; r < r1 - r0; r += kThreads) {
        const uint64_t units =
            __float_as_uint(sums[r].log_h) | static_cast<uint64_t>(__float_as_uint(sums[r].log_l)) << 32;
        const double l = units != 0 ? log(static_cast<double>(units) * kUnit) : 0.0;
        sums[r].log_h = units != 0 ? static_cast<float>(l) : INFINITY;
        sums[r].log_l = static_cast<float>(l - static_cast<float>(l));
    }
    __syncthreads();
    // ---- candidates: slot i of the request's (row, chunk, rank); an ended row has one ----
    const int64_t per_row = static_cast<int64_t>(S) * K, total = (r1 - r0) * per_row;
    auto candidate = [&](int64_t i, Candidate& c) -> bool {
        c.row = r0 + static_cast<int>(i / per_row);
        const int j = static_cast<int>(i - (c.row - r0) * per_row);
        const float score = p.scores[c.row];
        if (!(score > -INFINITY && score < INFINITY)) return false;
        if (p.ended != nullptr && p.ended[c.row] != 0) {
            c.s = {score, 0.f};
            c.key = static_cast<uint32_t>(~p.end_token);
            return j == 0;
        }
        const int chunk = j / K;
        c.key = reinterpret_cast<const uint64_t*>(head_of(c.row, chunk) + sizeof(ChunkHead))[j - chunk * K];
        const RowSum sum = sums[c.row - r0];
        if (c.key == 0 || sum.log_h == INFINITY) return false;
        // score + ((x - top) - log)
        const float x = value_of(static_cast<uint32_t>(c.key >> 32));
        c.s = two_add(two_add(two_sum(x, -sum.top), {-sum.log_h, -sum.log_l}), {score, 0.f});
        return true;
    };
    // (the score's float keeps the scores' order, so it serves as the threshold's key)
    auto key_of = [](Two s) -> uint32_t { return order_of(fmaxf(s.hi, -3.4028234e38f)); };
    uint32_t mine = kNothing;
    for (int64_t i = t; i < total; i += kThreads) {
        Candidate c;
        if (candidate(i, c)) mine = max(mine, key_of(c.s));
    }
    uint32_t top = __reduce_max_sync(0xffffffffu, mine);
    if (lane == 0) scratch[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) top = max(top, scratch[w]);
    const uint32_t cut = top == kNothing ? kNothing + 1 : threshold(mine, top, K, scratch);
    if (mine >= cut) {
        for (int64_t i = t; i < total; i += kThreads) {
            Candidate c;
            if (candidate(i, c) && key_of(c.s) >= cut) {
                const int n = atomicAdd(&list_n, 1);
                if (n < kList) list[n] = c;
            }
        }
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
        for (int i = t; i < n; i += kThreads) {
            const Candidate c = list[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += before(list[j], c);
            if (rank < K) put(rank, c);
        }
        if (t >= n && t < K) put(t, none);
        return;
    }
    // more than the list holds: one a round, the first behind the last one
    Candidate last{{INFINITY, 0.f}, 0, -1};
    for (int r = 0; r < K; ++r) {
        Candidate best = none;
        for (int64_t i = t; i < total; i += kThreads) {
            Candidate c;
            if (candidate(i, c) && before(last, c) && (best.row < 0 || before(c, best))) best = c;
        }
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

// Elements a thread holds.  More make longer loads and fewer lists; a small batch
// takes fewer, so that its chunks reach every SM.
int chunk_elems(int64_t rows, int vocab, int dtype, int sms) {
    const int most = dtype == PA_F32 ? 32 : 64;
    int ept = most;
    while (ept > 8 && rows * ((vocab + kThreads * ept - 1) / (kThreads * ept)) < 2ll * sms) ept /= 2;
    return ept;
}
int chunks_of(int vocab, int ept) { return (vocab + kThreads * ept - 1) / (kThreads * ept); }
int64_t chunk_bytes(int select) { return static_cast<int64_t>(sizeof(ChunkHead)) + 8ll * select; }

template <int DT, bool VEC>
cudaError_t launch_rows(const SelectParams& p, int ept, int grid, cudaStream_t s) {
    if (ept == 8) return launch_pdl(beam_rows_kernel<DT, 8, VEC>, grid, kThreads, 0, s, p);
    if (ept == 16) return launch_pdl(beam_rows_kernel<DT, 16, VEC>, grid, kThreads, 0, s, p);
    if constexpr (DT != PA_F32)
        if (ept == 64) return launch_pdl(beam_rows_kernel<DT, 64, VEC>, grid, kThreads, 0, s, p);
    return launch_pdl(beam_rows_kernel<DT, 32, VEC>, grid, kThreads, 0, s, p);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_beam_select_workspace_size(int32_t num_rows, int32_t vocab, int32_t num_select) {
    if (num_rows <= 0 || vocab <= 0 || num_select <= 0 || num_select > kMaxSelect) return 0;
    // (for the shortest chunks, which any device may take)
    const size_t chunks = static_cast<size_t>(num_rows) * chunks_of(vocab, 8);
    return static_cast<size_t>(num_rows) * sizeof(RowSum) + chunks * chunk_bytes(num_select);
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
    p.sums = static_cast<RowSum*>(workspace);
    p.chunks = static_cast<uint8_t*>(workspace) + static_cast<size_t>(num_rows) * sizeof(RowSum);
    p.row_stride = row_stride;
    p.allowed_stride = allowed_stride;
    p.vocab = vocab;
    p.num_rows = num_rows;
    p.num_requests = num_requests;
    p.select = num_select;
    p.end_token = end_token;
    const int ept = chunk_elems(num_rows, vocab, dtype, sms);
    p.chunks_per_row = chunks_of(vocab, ept);
    p.chunk_bytes = static_cast<int32_t>(chunk_bytes(num_select));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (num_rows > 0) {
        const int64_t grid = static_cast<int64_t>(num_rows) * p.chunks_per_row;
        if (grid > INT32_MAX) return PA_ERR_UNSUPPORTED;
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
