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
// Rows kernel: a block holds a chunk of one row in registers, read once.  The K-th
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
// 2^-40, which no order of addition changes.  Logarithms and s are binary64.
#include <cmath>

#include "common.cuh"
#include "launch.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxSelect = 64;
constexpr int kList = 1024;  // candidates a block ranks in shared memory
constexpr float kLog2e = 1.4426950408889634f;

// A row's log-sum-exp as its two terms: added up, a large maximum would take the
// logarithm's bits with it.
struct RowSum {
    double top;      // the row's largest logit
    double log_sum;  // log of the sum of exp(x - top); +inf: the row offers nothing
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

template <int DT>
struct Logits {  // 16-bit types, two to a register
    static constexpr int kVec = 8, kPerReg = 2;
    __device__ static float2 get(uint32_t w) { return kv_pair<DT>(w); }
    static constexpr uint32_t kNone = DT == PA_BF16 ? 0xff80u : 0xfc00u;  // -inf
};
template <>
struct Logits<PA_F32> {
    static constexpr int kVec = 4, kPerReg = 1;
    static constexpr uint32_t kNone = 0xff800000u;
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

// The largest threshold found in a few steps that at least `want` of the block's keys
// reach (fewer than want are above kNothing: the least that all of those reach).  Keys
// that hold nothing are kNothing.  top: the block's largest key.  Stops early once no
// more than 1.5 want reach it.
__device__ __forceinline__ uint32_t threshold(uint32_t key, uint32_t top, int want) {
    uint32_t lo = kNothing + 1, hi = top;  // count(lo) >= want once that is known; the answer is in [lo, hi]
    if (__syncthreads_count(key > kNothing) <= want) return lo;
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

// EPT elements a thread.  VEC: every row is 16-byte aligned and each thread reads
// whole vectors; otherwise pairs of 16-bit elements (or single floats), with the rows'
// own alignment.  Which element goes to which thread does not depend on a row's
// address, so equal rows get equal sums.
template <int DT, int EPT, bool VEC>
__global__ void __launch_bounds__(kThreads)
beam_rows_kernel(const SelectParams p) {
    using L = Logits<DT>;
    constexpr int kRegs = EPT / L::kPerReg;
    constexpr int kGroupRegs = 8 / L::kPerReg;  // registers of eight elements
    constexpr int kGroups = EPT / 8;
    __shared__ uint64_t list[kList];
    __shared__ uint64_t scratch64[kThreads / 32];
    __shared__ float scratch[kThreads / 32];
    __shared__ int list_n;

    const int t = threadIdx.x;
    const int row = blockIdx.x / p.chunks_per_row, chunk = blockIdx.x - row * p.chunks_per_row;
    const int first = chunk * (kThreads * EPT);
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
    // ---- the chunk into registers ----
    uint32_t raw[kRegs];
    const uint32_t* bits = p.allowed == nullptr ? nullptr : p.allowed + row * p.allowed_stride;
    // element of register i (its first)
    auto index = [&](int i) -> int {
        if constexpr (VEC) {
            constexpr int kVecRegs = L::kVec / L::kPerReg;
            return first + ((i / kVecRegs) * kThreads + t) * L::kVec + (i % kVecRegs) * L::kPerReg;
        } else {
            return first + (i * kThreads + t) * L::kPerReg;
        }
    };
    if constexpr (VEC) {
        constexpr int kVecRegs = L::kVec / L::kPerReg;
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint8_t*>(p.logits) + row * p.row_stride * (16 / L::kVec));
#pragma unroll
        for (int j = 0; j < kRegs / kVecRegs; ++j) {
            const int i0 = first + (j * kThreads + t) * L::kVec;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (i0 + L::kVec <= p.vocab) {
                v = __ldcs(src + i0 / L::kVec);
            } else if (i0 < p.vocab) {
                // (the row's last, partly filled vector: past it the buffer may end)
                if constexpr (L::kPerReg == 2) {
                    const uint16_t* e = reinterpret_cast<const uint16_t*>(src) + i0;
                    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (i0 + k < p.vocab) w[k / 2] |= static_cast<uint32_t>(e[k]) << (16 * (k & 1));
                    v = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
                    const uint32_t* e = reinterpret_cast<const uint32_t*>(src) + i0;
                    v.x = e[0];
                    if (i0 + 1 < p.vocab) v.y = e[1];
                    if (i0 + 2 < p.vocab) v.z = e[2];
                }
            }
            raw[j * kVecRegs] = v.x;
            raw[j * kVecRegs + 1] = v.y;
            raw[j * kVecRegs + 2] = v.z;
            raw[j * kVecRegs + 3] = v.w;
        }
    } else if constexpr (L::kPerReg == 2) {
        const uint16_t* e = static_cast<const uint16_t*>(p.logits) + row * p.row_stride;
        if ((reinterpret_cast<uintptr_t>(e) & 3u) == 0) {
#pragma unroll
            for (int i = 0; i < kRegs; ++i) {
                const int i0 = index(i);
                raw[i] = 0;
                if (i0 + 1 < p.vocab) raw[i] = __ldcs(reinterpret_cast<const uint32_t*>(e + i0));
                else if (i0 < p.vocab) raw[i] = e[i0];
            }
        } else {
            // a pair lies in two words: (e - 1 + i0, e + i0), (e + i0 + 1, e + i0 + 2)
#pragma unroll
            for (int i = 0; i < kRegs; ++i) {
                const int i0 = index(i);
                raw[i] = 0;
                if (i0 > 0 && i0 + 2 < p.vocab) {
                    const uint32_t* w = reinterpret_cast<const uint32_t*>(e + i0 - 1);
                    raw[i] = __funnelshift_r(__ldcs(w), __ldg(w + 1), 16);
                } else if (i0 < p.vocab) {
                    raw[i] = e[i0];
                    if (i0 + 1 < p.vocab) raw[i] |= static_cast<uint32_t>(e[i0 + 1]) << 16;
                }
            }
        }
    } else {
        const uint32_t* e = static_cast<const uint32_t*>(p.logits) + row * p.row_stride;
#pragma unroll
        for (int i = 0; i < kRegs; ++i) {
            const int i0 = index(i);
            raw[i] = i0 < p.vocab ? __ldcs(e + i0) : 0u;
        }
    }
    // what the row does not have or may not take: -inf
    const bool whole = first + kThreads * EPT <= p.vocab;
    if (!whole || bits != nullptr) {
#pragma unroll
        for (int i = 0; i < kRegs; ++i) {
            const int i0 = index(i);
            // (the pair's two bits lie in one word: i0 is even)
            uint32_t on = i0 < p.vocab ? ~0u : 0u;
            if (bits != nullptr && i0 < p.vocab) on = __ldg(bits + (i0 >> 5)) >> (i0 & 31);
            if constexpr (L::kPerReg == 2) {
                if (i0 + 1 >= p.vocab) on &= 1u;
                if (!(on & 1u)) raw[i] = (raw[i] & 0xffff0000u) | L::kNone;
                if (!(on & 2u)) raw[i] = (raw[i] & 0xffffu) | (L::kNone << 16);
            } else {
                if (!(on & 1u)) raw[i] = L::kNone;
            }
        }
    }
    auto element = [&](int i) -> float {  // i-th of the thread's EPT
        if constexpr (L::kPerReg == 2) {
            const float2 f = L::get(raw[i / 2]);
            return i & 1 ? f.y : f.x;
        } else {
            return __uint_as_float(raw[i]);
        }
    };
    auto token = [&](int i) -> int { return index(i / L::kPerReg) + i % L::kPerReg; };
    // ---- maxima: of every eight elements, the thread's, the block's ----
    float gmax[kGroups], mine = -INFINITY;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        gmax[g] = element(8 * g);
#pragma unroll
        for (int i = 1; i < 8; ++i) gmax[g] = max_nan(gmax[g], element(8 * g + i));
        mine = max_nan(mine, gmax[g]);
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
    const uint32_t cut = threshold(order_of(mine), order_of(top), p.select);
    const float cut_v = value_of(cut);
    // ---- the list of what reaches the threshold; the sum of the rest ----
    // exp(x - top): the difference first, which is exact or nearly so (a product with
    // log2 e first would lose what a large common part of the logits takes)
    auto exp_of = [&](float x) -> float { return exp2_approx((x - top) * kLog2e); };
    float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        if (gmax[g] >= cut_v) {
#pragma unroll
            for (int i = 8 * g; i < 8 * g + 8; ++i) {
                const float x = element(i);
                if (x >= cut_v) {
                    const int at = atomicAdd(&list_n, 1);
                    if (at < kList)
                        list[at] = (static_cast<uint64_t>(order_of(x)) << 32) | static_cast<uint32_t>(~token(i));
                } else {
                    sum0 += exp_of(x);
                }
            }
        } else {
#pragma unroll
            for (int i = 8 * g; i < 8 * g + 8; i += 2) {
                sum0 += exp_of(element(i));
                sum1 += exp_of(element(i + 1));
            }
        }
    }
    uint64_t units = static_cast<uint64_t>(__float2ll_rn((sum0 + sum1) * 1099511627776.f));
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
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                const float x = element(i);
                const uint64_t k = (static_cast<uint64_t>(order_of(x)) << 32) | static_cast<uint32_t>(~token(i));
                if (x > -INFINITY && k < last && k > best) best = k;
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
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const float x = element(i);
            const uint64_t k = (static_cast<uint64_t>(order_of(x)) << 32) | static_cast<uint32_t>(~token(i));
            if (x > -INFINITY && k < last)
                units += static_cast<uint64_t>(__float2ll_rn(exp_of(x) * 1099511627776.f));
        }
    }
    units = block_sum(units, scratch64);
    if (t == 0) *head = {units, top, 0};
}

struct Candidate {
    double s;
    uint64_t key;  // the logit's order, then the token's complement
    int32_t row;
};
// c stands before d: by score, then row; of one row by logit (a large maximum can take
// the difference from their scores), then token
__device__ __forceinline__ bool before(const Candidate& c, const Candidate& d) {
    if (c.s != d.s) return c.s > d.s;
    if (c.row != d.row) return c.row < d.row;
    return c.key > d.key;
}

// One block a request.
__global__ void __launch_bounds__(kThreads)
beam_requests_kernel(const SelectParams p) {
    __shared__ Candidate list[kList];
    __shared__ Candidate warp_best[kThreads / 32];
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
    // ---- each row's log-sum-exp: a warp takes a row ----
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
        double log_sum = INFINITY;
        if (bad) {
            if (lane == 0) report(p.status, PA_ERR_INVALID_ARG);
        } else if (top > -INFINITY) {
            uint64_t units = 0;
            for (int i = lane; i < S * K; i += 32) {
                const int c = i / K;
                const uint64_t k = reinterpret_cast<const uint64_t*>(head_of(row, c) + sizeof(ChunkHead))[i - c * K];
                if (k != 0) units += exp_units(value_of(static_cast<uint32_t>(k >> 32)), top);
            }
            // (a chunk's units count against its own maximum)
            double rest = 0.0;
            for (int c = lane; c < S; c += 32) {
                const ChunkHead h = *reinterpret_cast<const ChunkHead*>(head_of(row, c));
                if (h.sum != 0)
                    rest += static_cast<double>(h.sum) * (static_cast<double>(exp_units(h.top, top)) * kUnit);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                units += __shfl_xor_sync(0xffffffffu, units, o);
                rest += __shfl_xor_sync(0xffffffffu, rest, o);
            }
            log_sum = log((static_cast<double>(units) + rest) * kUnit);
        }
        if (lane == 0) p.sums[row] = {top, log_sum};
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
            c.s = score;
            c.key = static_cast<uint32_t>(~p.end_token);
            return j == 0;
        }
        const int chunk = j / K;
        c.key = reinterpret_cast<const uint64_t*>(head_of(c.row, chunk) + sizeof(ChunkHead))[j - chunk * K];
        const RowSum sum = p.sums[c.row];
        if (c.key == 0 || sum.log_sum == INFINITY) return false;
        const double x = value_of(static_cast<uint32_t>(c.key >> 32));
        c.s = static_cast<double>(score) + ((x - sum.top) - sum.log_sum);
        return true;
    };
    // (a score's float keeps the scores' order, so it serves as the threshold's key)
    auto key_of = [](double s) -> uint32_t { return order_of(fmaxf(static_cast<float>(s), -3.4028234e38f)); };
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
    const uint32_t cut = top == kNothing ? kNothing + 1 : threshold(mine, top, K);
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
        p.scores_out[out0 + rank] = static_cast<float>(c.s);
        p.rows_out[out0 + rank] = c.row;
        p.tokens_out[out0 + rank] = c.row < 0 ? -1 : static_cast<int32_t>(~static_cast<uint32_t>(c.key));
    };
    const Candidate none{-INFINITY, 0, -1};
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
    Candidate last{INFINITY, 0, -1};
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
            const Candidate c{__shfl_xor_sync(0xffffffffu, best.s, o), __shfl_xor_sync(0xffffffffu, best.key, o),
                              __shfl_xor_sync(0xffffffffu, best.row, o)};
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
    if (num_select > kMaxSelect) return PA_ERR_UNSUPPORTED;
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
