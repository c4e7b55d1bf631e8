// Varlen (prefill / mixed) attention over the paged KV cache on the
// 5th-generation tensor cores (tcgen05, accumulators in tensor memory).
//
// "Paged 어텐션" (data-sketchers.com transformers paged-attention wiki),
// Varlen 경로: a batch of sequences of different lengths is indexed by the
// cumulative lengths cu_seq_lens_q / cu_seq_lens_k (bounded by max_seqlen_q /
// max_seqlen_k); here the keys and values come from the paged cache through
// block_table (Decode 경로) instead of packed K/V tensors.
// "Как работает paged attention? (детально)" 5.1: attention runs block by
// block over the physical blocks, with the causal mask applied per block.
// Softmax by max subtraction as in the vLLM PagedAttention design doc
// (section Softmax), kept online across key tiles.
//
// Work item = (sequence, tile of TQ = 128/G query tokens, KV head): its 128
// rows are the G query heads of the KV head for TQ tokens (row = t*G + g), so
// one key/value tile serves the whole GQA group.  Items are sorted by their
// key-tile count and dealt to the persistent blocks in snake order.  Per
// item, key tiles of 128 keys stream through a 3-stage K ring and a 2-stage
// V ring:
//   warps 0, 2  load pages with TMA tensor copies (128B swizzle), through the
//               block table (or 3-D boxes of packed K/V): warp 0 the K ring,
//               warp 2 the V ring;
//   warp 3      loads each item's 128 query rows into shared memory in the
//               layout of a K tile once the previous item's last QK is done
//               (two 3-D TMA boxes; at the batch's end 16-byte asynchronous
//               copies, zero past the sequence);
//   warp 1      allocates tensor memory and issues every MMA from one thread:
//               S[t & 1] = Q K(t)^T from shared memory, then
//               O[c] += P V(t) with the weights P written over S[t & 1]; two
//               O buffers (c alternates per item) let one item's epilogue run
//               beside the next item's first PV;
//   warps 4..7, two softmax warpgroups that split the 128 key columns of each
//   8..11       tile (a thread: 64 columns of one row, its tensor-memory
//               lane).  They take weights against a shared reference max and
//               vote at a barrier whether any row's sum would pass 2^64; only
//               then (and on an item's first tile) is the true max taken,
//               exchanged through shared memory, O rescaled in tensor memory
//               and the weights recomputed.  Weights go to tensor memory as
//               bf16 hi + lo (both truncated, ~16 bits together; two PV
//               passes) or one fp16.  An item's epilogue (O / l) is written
//               once the next item's first weights are out.
// Causal alignment is bottom-right: query i of a sequence with Lq queries and
// Lk keys sits at position Lk - Lq + i.  Every wait is bounded.
//
// Sliding window and sinks (pa_prefill_varlen_window): an item works on the
// sinks' blocks and those of its window as if they were all of its keys, so its
// tiles hold few keys that no row sees (1028 seen of 1152 for an item past the
// window's start: a window of 1024, 4 sinks, 32 queries, blocks of 16).  Bound by the
// softmax warps' chain of about 2330 cycles a tile (scores 240, exponentials and vote
// 1100, weights stored 580; beside it the issuing thread spends 970 on PV, two passes
// of bf16 weights, and 390 on QK) and some 5000 cycles an item: its first tile's true
// maximum (1860), the previous item's output.  On one GB300 eight chunks of 512 to
// 2048 queries on up to 4096 cached tokens (32/8 heads, bf16, window 1024, 4 sinks) take
// 223 us, 679 TFLOP/s of visible pairs; one prompt of 8192 tokens, window 2048, 280 us,
// 866 TFLOP/s; in fp16, one PV pass, 196 and 243 us.
#include <cmath>
#include <type_traits>

#include "tcgen05.cuh"

namespace pa {
namespace {

constexpr int kStages = 3;           // depth of the K ring
constexpr int kStagesV = 2;          // depth of the V ring
constexpr int kThreads = 384;        // 12 warps
constexpr int kSoftWarp0 = 4;        // softmax warpgroups = warps 4..7 and 8..11
constexpr uint32_t kTmemCols = 512;
// tensor-memory columns: S[b] (fp32 scores of the key tiles t with t & 1 = b,
// later overwritten by the 16-bit weights P) and O[c] (fp32 accumulators of
// the items with key tiles, c = their count & 1: one item's O is written out
// while the next item's first PV goes to the other)
constexpr uint32_t kColS = 0;    // S[b] at b * kBN
constexpr uint32_t kColO = 256;  // O[c] at kColO + c * kD

// shared memory layout (bytes from the 1 KB-aligned base)
constexpr int kOffK = 0;                       // K ring
constexpr int kOffV = kOffK + kStages * kTileBytes;  // V ring
constexpr int kOffQ = kOffV + kStagesV * kTileBytes; // the item's 128 query rows, laid out like a K tile
constexpr int kOffBar = kOffQ + kTileBytes;
constexpr int kNumBars = 2 * kStages + 2 * kStagesV + 3 * 2 + 3;
constexpr int kOffMisc = kOffBar + kNumBars * 8;
constexpr int kOffXch = kOffMisc + 64;                   // [2 slots][2 warpgroups][128 rows] floats
constexpr int kOffPend = kOffXch + 2 * 2 * kRows * 4;  // [256] int64 row offsets, then [256] float row sums
constexpr int kItemCache = 64;                          // a CTA's first items, worked out once
constexpr int kOffItems = kOffPend + 256 * 12;          // [kItemCache] Work
constexpr int kSmemBytes = kOffItems + kItemCache * 32;
constexpr int kMaxSeqs = 6144;                           // prefix of query tiles: (B + 1) ints

struct PrefillParams {
    void* out;
    const uint16_t* q;  // NULL (pa_prefill_test_wait_timeout): no copy is issued, every wait runs out
    const int32_t* block_table;
    const int32_t* cu_q;
    const int32_t* cu_k;
    int32_t* status;
    int64_t num_blocks;
    int32_t block_size;
    int32_t num_kv_heads;
    int32_t num_heads;
    int32_t group;  // num_heads / num_kv_heads
    int32_t tq;     // query tokens per item (128 / group)
    int32_t num_seqs;
    int32_t max_blocks;
    int32_t max_q;
    int32_t max_k;
    int32_t causal;
    float scale_log2;  // scale * log2(e)
    int64_t total_k;   // packed K/V: rows of K and V (Σ key lengths); -1 for the paged cache
    int32_t order_cap; // query tiles the shared-memory work order holds (set by the launch)
    int32_t q_rows;    // token extent of the query tensor map: min(num_seqs * max_seqlen_q, INT32_MAX)
};

// Sliding window (pa_prefill_varlen_window): a query sees the last `window`
// positions up to its own and the first `sinks`, which lie in `head` blocks.
// (Fields of their own: three more in the plain launches' parameters made the
// compiler spill 20 bytes more in their softmax.)
struct WindowParams : PrefillParams {
    int32_t window, sinks, head;
    const uint16_t* k_cache;  // (redo_rows)
    const uint16_t* v_cache;
};
template <bool WIN>
using ParamsOf = std::conditional_t<WIN, WindowParams, PrefillParams>;
template <bool WIN>
__device__ __forceinline__ int sinks_of(const ParamsOf<WIN>& p) {
    if constexpr (WIN) return p.sinks;
    else return 0;
}
template <bool WIN>
__device__ __forceinline__ int head_of(const ParamsOf<WIN>& p) {
    if constexpr (WIN) return p.head;
    else return 0;
}
// first position that a query at position `pos` sees through the window
template <bool WIN>
__device__ __forceinline__ int first_key(const ParamsOf<WIN>& p, int pos) {
    if constexpr (WIN) return max(0, pos - p.window + 1);
    else return 0;
}

// lengths of sequence b; false if they break the stated bounds
__device__ __forceinline__ bool seq_lens_ok(const PrefillParams& p, int b, int& lq, int& lk) {
    const int q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1);
    const int k0 = __ldg(p.cu_k + b);
    const int k1 = __ldg(p.cu_k + b + 1);
    lq = q1 - q0;
    lk = k1 - k0;
    const bool fits = p.total_k >= 0 ? (k0 >= 0 && static_cast<int64_t>(k1) <= p.total_k)
                                     : static_cast<int64_t>(lk) <= static_cast<int64_t>(p.max_blocks) * p.block_size;
    return lq >= 0 && lk >= 0 && lq <= p.max_q && lk <= p.max_k && fits;
}

struct Work {
    int b, i0, kvh, lq, lk, ntiles;
    int skip;  // sliding window: blocks left out between the sinks' and the window's
    int q0;  // cu_q[b]: the sequence's first query row
};
static_assert(sizeof(Work) == 32, "the item cache holds 32-byte entries");

// What an item's queries i0 .. min(i0 + tq, lq) - 1 see lies in keys 0 .. kend-1
// and, with a sliding window (WIN), from these without the blocks between the
// sinks' `head` and the window of the item's first query: the item works on the
// blocks that are left as if they were all, position v standing for v + skip *
// block_size past the sinks' blocks.  A row then sees v < sinks and lo <= v < lim
// with its own lo and lim in those positions (skip > 0: the sinks' last block
// ends at or before every row's lo).
template <bool WIN>
__device__ __forceinline__ int key_tiles(const ParamsOf<WIN>& p, int i0, int lq, int lk, int& skip) {
    int kend = lk;
    if (WIN || p.causal) kend = min(lk, lk - lq + min(i0 + p.tq, lq));
    skip = 0;
    if constexpr (WIN) {
        skip = max(0, first_key<WIN>(p, lk - lq + i0) / p.block_size - p.head);
        kend -= skip * p.block_size;
    }
    return kend > 0 ? (kend + kBN - 1) / kBN : 0;
}

// Work order.  An item's cost is its number of key tiles, which under the
// causal mask grows along a sequence's query tiles and differs widely between
// sequences.  When the query tiles fit the shared-memory order array, every
// CTA sorts them by cost class (64 classes, most key tiles first, ties in
// list order) and deals the items out in snake order (snake_item): the
// CTAs' totals then stay within about 1 % of each other on a mixed batch,
// where round-robin in sequence order left the busiest 11 % above the mean.
// Otherwise the items keep sequence order.
__device__ __forceinline__ int tile_seq(const PrefillParams& p, const int32_t* prefix, int tile) {
    int lo = 0, hi = p.num_seqs - 1;  // largest b with prefix[b] <= tile
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= tile) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <bool WIN>
__device__ __forceinline__ int tile_class(const ParamsOf<WIN>& p, const int32_t* prefix, int tile) {
    const int b = tile_seq(p, prefix, tile);
    int lq, lk;
    seq_lens_ok(p, b, lq, lk);
    const int i0 = (tile - prefix[b]) * p.tq;
    int skip;
    int most = p.max_k;
    if constexpr (WIN) {
        // (the most keys of an item: the sinks' blocks, the window, the item's
        // other queries, the rest of the window's first block)
        const int64_t span = static_cast<int64_t>(p.head + 1) * p.block_size + p.window + p.tq;
        most = static_cast<int>(min(span, static_cast<int64_t>(most)));
    }
    const int maxt = (most + kBN - 1) / kBN;
    const int nt = min(maxt, key_tiles<WIN>(p, i0, lq, lk, skip));
    return 63 - static_cast<int>((static_cast<int64_t>(nt) * 64) / (maxt + 1));  // 0 = most key tiles
}

// Stable counting sort of the n query tiles by class: each warp counts a
// contiguous chunk (lanes of equal class found by match.any), warp 0 turns
// the [warp][class] counts into class-major offsets, each warp then places its
// chunk in order.  All threads of the block take part; hist holds 12*64 ints.
template <bool WIN>
__device__ void build_tile_order(const ParamsOf<WIN>& p, const int32_t* prefix, int n, int32_t* order,
                                 int32_t* hist) {
    constexpr int NW = kThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunk = ((n + NW - 1) / NW + 31) & ~31;
    const int t0 = warp * chunk, t1 = min(n, t0 + chunk);
    int32_t* h = hist + warp * 64;
    h[lane] = 0;
    h[lane + 32] = 0;
    __syncwarp();
    for (int c0 = t0; c0 < t1; c0 += 32) {
        const int t = c0 + lane;
        const int key = t < t1 ? tile_class<WIN>(p, prefix, t) : 64;
        const unsigned same = __match_any_sync(0xffffffffu, key);
        if (t < t1 && lane == __ffs(same) - 1) h[key] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    if (warp == 0) {
        int tot0 = 0, tot1 = 0;
        for (int w = 0; w < NW; ++w) {
            tot0 += hist[w * 64 + 2 * lane];
            tot1 += hist[w * 64 + 2 * lane + 1];
        }
        int incl = tot0 + tot1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        int base0 = incl - tot0 - tot1, base1 = incl - tot1;
        for (int w = 0; w < NW; ++w) {
            const int x0 = hist[w * 64 + 2 * lane], x1 = hist[w * 64 + 2 * lane + 1];
            hist[w * 64 + 2 * lane] = base0;
            hist[w * 64 + 2 * lane + 1] = base1;
            base0 += x0;
            base1 += x1;
        }
    }
    __syncthreads();
    for (int c0 = t0; c0 < t1; c0 += 32) {
        const int t = c0 + lane;
        const int key = t < t1 ? tile_class<WIN>(p, prefix, t) : 64;
        const unsigned same = __match_any_sync(0xffffffffu, key);
        if (t < t1) order[h[key] + __popc(same & ((1u << lane) - 1u))] = t;
        __syncwarp();
        if (t < t1 && lane == __ffs(same) - 1) h[key] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
}

template <bool WIN>
__device__ __forceinline__ Work work_item(const ParamsOf<WIN>& p, const int32_t* prefix, const int32_t* order,
                                          int item) {
    Work w;
    int tile_id = item / p.num_kv_heads;
    w.kvh = item - tile_id * p.num_kv_heads;
    if (order != nullptr) tile_id = order[tile_id];
    int lo = 0, hi = p.num_seqs - 1;  // largest b with prefix[b] <= tile_id
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= tile_id) lo = mid;
        else hi = mid - 1;
    }
    w.b = lo;
    seq_lens_ok(p, lo, w.lq, w.lk);
    w.q0 = __ldg(p.cu_q + lo);
    w.i0 = (tile_id - prefix[lo]) * p.tq;
    w.ntiles = key_tiles<WIN>(p, w.i0, w.lq, w.lk, w.skip);
    return w;
}

// Scores of keys that are not seen: those from vis on and (WIN) [hid0, hid1).
template <bool WIN>
__device__ __forceinline__ void hide_keys(float (&e)[64], int vis, int hid0, int hid1) {
    if constexpr (WIN) {
        if (vis < 64) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
                if (i >= vis) e[i] = -INFINITY;
        }
        if (hid0 < hid1) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
                if (i >= hid0 && i < hid1) e[i] = -INFINITY;
        }
    } else if (vis < 64) {
#pragma unroll
        for (int i = 0; i < 64; ++i)
            if (i >= vis) e[i] = -INFINITY;
    }
}

// Sliding window: rows whose O came out infinite or NaN although the sum of their
// weights is finite, from the definition.  In a tile's product a weight of zero
// still multiplies the value of a key that only other rows of the item see, so a
// value there that is not finite reaches them all; and values near the type's end
// can overflow under weights that are not divided by their sum yet.  Such rows are
// found in `out`, and a warp takes one at a time, four columns a lane.  First the
// values that the row does see: where one is not finite it is the output, no weight
// being zero.  For what that leaves, the scores of 32 keys, one a lane, once for their
// maximum and sum and again for the values under divided weights.  qs: 128 floats of
// this warp in shared memory.  (8192 tokens, 32/8 heads, window 2048: one infinite
// value in one KV head 10 ms in place of 0.28, one in every block 22 ms.)
template <int DT>
__device__ __forceinline__ void redo_rows(const WindowParams& p, const int32_t* prefix, const int32_t* order,
                                          int n_items, float* qs) {
    const int lane = threadIdx.x & 31;
    for (int rnd = 0, item; (item = snake_item(rnd, n_items)) >= 0; ++rnd) {
        const Work w = work_item<true>(p, prefix, order, item);
        const int32_t* table = p.block_table + static_cast<int64_t>(w.b) * p.max_blocks;
        for (int r = threadIdx.x >> 5; r < kRows; r += kThreads / 32) {
            const int qi = w.i0 + r / p.group, head = w.kvh * p.group + r % p.group;
            if (qi >= w.lq) break;
            const int64_t at = (static_cast<int64_t>(w.q0 + qi) * p.num_heads + head) * kD + 4 * lane;
            uint2* dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at);
            const float2 o01 = kv_pair<DT>(dst->x), o23 = kv_pair<DT>(dst->y);
            const bool good = fabsf(o01.x) < INFINITY && fabsf(o01.y) < INFINITY && fabsf(o23.x) < INFINITY &&
                              fabsf(o23.y) < INFINITY;
            if (__all_sync(0xffffffffu, good)) continue;
            // the row's n keys: the sinks before its window, then the window
            const int pos = w.lk - w.lq + qi, lo = first_key<true>(p, pos), first = min(p.sinks, lo);
            const int n = first + pos + 1 - lo;
            // key number v's row in the cache, -1: in a block that the loaders reported
            auto row_of = [&](int v) -> int64_t {
                const int j = v < first ? v : v - first + lo;
                const int id = __ldg(table + j / p.block_size);
                if (id < 0 || id >= p.num_blocks) return -1;
                return ((static_cast<int64_t>(id) * p.num_kv_heads + w.kvh) * p.block_size + j % p.block_size) * kD;
            };
            // its values of this lane's columns (0 for none; no branch, so that loads run ahead)
            auto value = [&](int64_t row, float (&x)[4]) {
                const uint2 raw = *reinterpret_cast<const uint2*>(p.v_cache + max(row, int64_t{0}) + 4 * lane);
                const float2 a = kv_pair<DT>(raw.x), b = kv_pair<DT>(raw.y);
                x[0] = row < 0 ? 0.f : a.x;
                x[1] = row < 0 ? 0.f : a.y;
                x[2] = row < 0 ? 0.f : b.x;
                x[3] = row < 0 ? 0.f : b.y;
            };
            // sums of the values that are not finite: one such value, or NaN
            float odd[4] = {0.f, 0.f, 0.f, 0.f};
            for (int v = 0; v < n; v += 32) {
                const int64_t mine = v + lane < n ? row_of(v + lane) : -1;
#pragma unroll 8
                for (int i = 0; i < 32; ++i) {
                    float x[4];
                    value(__shfl_sync(0xffffffffu, mine, i), x);
#pragma unroll
                    for (int c = 0; c < 4; ++c) odd[c] += fabsf(x[c]) < INFINITY ? 0.f : x[c];
                }
            }
            const float was[4] = {o01.x, o01.y, o23.x, o23.y};
            float acc[4];
            bool left = false;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                acc[c] = odd[c] == 0.f ? was[c] : odd[c];
                left |= odd[c] == 0.f && !(fabsf(was[c]) < INFINITY);
            }
            if (!__any_sync(0xffffffffu, left)) {
                *dst = make_uint2(pack2<DT>(acc[0], acc[1]), pack2<DT>(acc[2], acc[3]));
                continue;
            }
            const uint2 qw = *reinterpret_cast<const uint2*>(p.q + at);
            const float2 q01 = kv_pair<DT>(qw.x), q23 = kv_pair<DT>(qw.y);
            __syncwarp();
            *reinterpret_cast<float4*>(qs + 4 * lane) = make_float4(q01.x, q01.y, q23.x, q23.y);
            __syncwarp();
            auto score = [&](int v, int64_t& row) -> float {
                row = v < n ? row_of(v) : -1;
                if (row < 0) return -INFINITY;
                const uint4* k = reinterpret_cast<const uint4*>(p.k_cache + row);
                float sc = 0.f;
#pragma unroll 4
                for (int c = 0; c < kD / 8; ++c) {
                    const uint4 x = k[c];
                    const float4 a = *reinterpret_cast<const float4*>(qs + 8 * c);
                    const float4 b = *reinterpret_cast<const float4*>(qs + 8 * c + 4);
                    const float2 k0 = kv_pair<DT>(x.x), k1 = kv_pair<DT>(x.y), k2 = kv_pair<DT>(x.z), k3 = kv_pair<DT>(x.w);
                    sc = fmaf(a.x, k0.x, fmaf(a.y, k0.y, fmaf(a.z, k1.x, fmaf(a.w, k1.y, sc))));
                    sc = fmaf(b.x, k2.x, fmaf(b.y, k2.y, fmaf(b.z, k3.x, fmaf(b.w, k3.y, sc))));
                }
                return sc * p.scale_log2;
            };
            auto weight = [](float sc, float m) { return sc == -INFINITY ? 0.f : ex2(sc - m); };
            int64_t row;
            float m = -INFINITY, l = 0.f;
            for (int v = lane; v < n; v += 32) {
                const float sc = score(v, row), top = fmaxf(m, sc);
                l = l * weight(m, top) + weight(sc, top);
                m = top;
            }
            float top = m;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            l *= weight(m, top);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
            const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[c] = 0.f;
            for (int v = 0; v < n; v += 32) {
                const float mine = weight(score(v + lane, row), top) * inv;
#pragma unroll 8
                for (int i = 0; i < 32; ++i) {
                    const float wt = __shfl_sync(0xffffffffu, mine, i);
                    float x[4];
                    value(__shfl_sync(0xffffffffu, row, i), x);
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[c] = fmaf(wt, x[c], acc[c]);
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[c] = odd[c] == 0.f ? acc[c] : odd[c];
            *dst = make_uint2(pack2<DT>(acc[0], acc[1]), pack2<DT>(acc[2], acc[3]));
        }
    }
}

// PACKED: K and V are contiguous [Σk][num_kv_heads][head_size] tensors indexed
// by cu_seq_lens_k (no cache, no block table); otherwise the paged cache.
// WIN: causal with a sliding window and sinks (an instantiation of its own, so
// that the others' softmax carries no second mask).
template <int DT, bool PACKED, bool WIN>
__global__ void __launch_bounds__(kThreads, 1)
paged_prefill_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                        const __grid_constant__ CUtensorMap map_q,
                        const ParamsOf<WIN> p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // 128B-swizzled tiles need 1 KB alignment; the launch adds 1 KB of slack
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sK = smem + kOffK;
    uint8_t* sV = smem + kOffV;
    uint8_t* sQ = smem + kOffQ;
    const uint32_t bar0 = smem_addr(smem + kOffBar);
    const uint32_t k_full = bar0;                       // [kStages] TMA bytes of a K tile
    const uint32_t k_empty = k_full + 8 * kStages;      // [kStages] MMA commit after QK
    const uint32_t v_full = k_empty + 8 * kStages;      // [kStagesV] TMA bytes of a V tile
    const uint32_t v_empty = v_full + 8 * kStagesV;     // [kStagesV] MMA commit after PV
    const uint32_t s_full = v_empty + 8 * kStagesV;     // [2] MMA commit after QK into S[b]
    const uint32_t p_full = s_full + 16;           // [2] the 8 softmax warps: P[b] written
    const uint32_t o_done = p_full + 16;           // [2] MMA commit after PV number g, on o_done[g & 1]
    const uint32_t q_full = o_done + 16;           // the query loader warp: an item's Q in shared memory
    const uint32_t q_empty = q_full + 8;           // MMA commit after an item's last QK
    const uint32_t mma_done = q_empty + 8;         // MMA commit at the very end
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
    volatile int* snap = reinterpret_cast<volatile int*>(smem + kOffMisc + 8);  // [2] abort snapshots
    [[maybe_unused]] volatile int* redo = reinterpret_cast<volatile int*>(smem + kOffMisc + 16);  // redo_rows has work
    float* xch = reinterpret_cast<float*>(smem + kOffXch);
    int64_t* pend_off = reinterpret_cast<int64_t*>(smem + kOffPend);        // pending epilogue: out offset (-1: no row)
    float* pend_l = reinterpret_cast<float*>(smem + kOffPend + 256 * 8);     // and partial row sum, per thread
    int32_t* prefix = reinterpret_cast<int32_t*>(smem + kSmemBytes);  // B + 1 ints past the fixed layout
    __shared__ int32_t scan_scratch[kThreads / 32];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int B = p.num_seqs;

    pdl_wait();
    pdl_trigger();
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(k_full + 8 * s, 1);
            mbar_init(k_empty + 8 * s, 1);
        }
        for (int s = 0; s < kStagesV; ++s) {
            mbar_init(v_full + 8 * s, 1);
            mbar_init(v_empty + 8 * s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(s_full + 8 * s, 1);
            mbar_init(p_full + 8 * s, 8);
            mbar_init(o_done + 8 * s, 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        *redo = 0;
        snap[0] = 0;
        snap[1] = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }

    // ---- per-sequence prefix of query tiles ----
    {
        const int chunk = (B + kThreads - 1) / kThreads;
        const int b0 = tid * chunk, b1 = min(B, b0 + chunk);
        int local = 0;
        for (int b = b0; b < b1; ++b) {
            int lq, lk;
            if (seq_lens_ok(p, b, lq, lk)) local += (lq + p.tq - 1) / p.tq;
            else report(p.status, PA_ERR_INVALID_ARG);
        }
        int v = local;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += n;
        }
        if (lane == 31) scan_scratch[warp] = v;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (tid == 0) {
            int run = 0;
            for (int w = 0; w < kThreads / 32; ++w) {
                const int x = scan_scratch[w];
                scan_scratch[w] = run;
                run += x;
            }
            prefix[B] = run;
        }
        __syncthreads();
        int run = scan_scratch[warp] + v - local;
        for (int b = b0; b < b1; ++b) {
            prefix[b] = run;
            int lq, lk;
            if (seq_lens_ok(p, b, lq, lk)) run += (lq + p.tq - 1) / p.tq;
        }
        __syncthreads();
    }
    // ---- work order of the query tiles ----
    const int32_t* order = nullptr;
    // (window: no more items than blocks need no order; sorting them took 1.3 us
    // of a small batch's 11)
    if (p.order_cap > 0 && prefix[B] <= p.order_cap &&
        (!WIN || static_cast<int64_t>(prefix[B]) * p.num_kv_heads > gridDim.x)) {
        int32_t* ord = prefix + B + 1;
        build_tile_order<WIN>(p, prefix, prefix[B], ord, ord + p.order_cap);
        order = ord;
    }
    const uint32_t tmem = uniform(*tmem_slot);
    const int n_items = prefix[B] * p.num_kv_heads;
    // this CTA's first kItemCache items, worked out once: every role's item
    // loop reads them from here (item_work) instead of searching the tile
    // prefix and reading the sequence lengths at each item boundary
    Work* item_cache = reinterpret_cast<Work*>(smem + kOffItems);
    if (tid < kItemCache) {
        const int item = snake_item(tid, n_items);
        if (item >= 0) item_cache[tid] = work_item<WIN>(p, prefix, order, item);
    }
    __syncthreads();
    auto item_work = [&](int rnd, int item) -> Work {
        return rnd < kItemCache ? item_cache[rnd] : work_item<WIN>(p, prefix, order, item);
    };
    if (warp == 0 || warp == 2) {
        // ------------------------------- loaders -------------------------------
        // K (warp 0) and V (warp 2) have rings and loader warps of their own: a
        // K stage is free again once its QK is done, long before the PV of the
        // same tile has used V, and each warp issues only half of a tile's
        // copies (a tile of block-size-16 pages is 16 copies of K and 16 of V,
        // issued lane by lane).
        const int kv = warp == 0 ? 0 : 1;
        const uint32_t full0 = kv == 0 ? k_full : v_full;
        const uint32_t empty0 = kv == 0 ? k_empty : v_empty;
        const uint32_t ring = smem_addr(kv == 0 ? sK : sV);
        const CUtensorMap* map = kv == 0 ? &map_k : &map_v;
        const uint32_t nst = kv == 0 ? kStages : kStagesV;  // ring depth
        uint32_t fill = 0, stage = 0, phase = 0;
        bool ok = p.q != nullptr;
        if constexpr (PACKED) {
            // a tile is 128 consecutive rows of one KV head: one 3-D box per
            // 64-column half (rows past the tensor read as zero; rows past the
            // sequence are masked / zeroed by the softmax warps)
            for (int rnd = 0, item; ok && (item = snake_item(rnd, n_items)) >= 0; ++rnd) {
                const Work w = item_work(rnd, item);
                const int row0 = __ldg(p.cu_k + w.b);
                for (int t = 0; t < w.ntiles && ok; ++t) {
                    const uint32_t full = full0 + 8 * stage;
                    if (lane == 0) ok = mbar_wait(empty0 + 8 * stage, phase ^ 1u, p.status, abort_flag);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_expect_tx(full, kTileBytes);
                        const uint32_t dst = ring + stage * kTileBytes;
                        tma_load_3d(dst, map, 0, w.kvh, row0 + t * kBN, full);
                        tma_load_3d(dst + kBlkBytes, map, 64, w.kvh, row0 + t * kBN, full);
                    }
                    __syncwarp();
                    ++fill;
                    if (++stage == nst) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        } else {
            const int ppt = kBN / p.block_size;  // pages per tile (2, 4 or 8)
            for (int rnd = 0, item; ok && (item = snake_item(rnd, n_items)) >= 0; ++rnd) {
                const Work w = item_work(rnd, item);
                const int32_t* bt_row = p.block_table + static_cast<int64_t>(w.b) * p.max_blocks;
                // page ids come in batches of 32 (one per lane, -1: past Lk, -2:
                // bad id), so the table's latency is paid once per batch
                const int pages = (w.ntiles * kBN + p.block_size - 1) / p.block_size;
                int32_t id = -1;
                for (int t = 0; t < w.ntiles && ok; ++t) {
                    const int pg0 = t * ppt;  // first page of this tile
                    if ((pg0 & 31) == 0) {
                        const int pg = pg0 + lane;
                        const int entry = WIN && pg >= head_of<WIN>(p) ? pg + w.skip : pg;
                        id = -1;
                        if (pg < pages && entry * p.block_size < w.lk) {
                            id = __ldg(bt_row + entry);
                            if (id < 0 || id >= p.num_blocks) {
                                // both loader warps read the id; one reports it
                                if (kv == 0) report(p.status, PA_ERR_BAD_BLOCK);
                                id = -2;
                            }
                        }
                    }
                    // lane k < ppt holds the id of page k of this tile
                    const int my_id = __shfl_sync(0xffffffffu, id, (pg0 + (lane & 7)) & 31);
                    const bool have = lane < ppt && my_id >= 0;
                    const uint32_t bytes =
                        static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, have))) * 2u * p.block_size * kD;
                    const int row = (my_id * p.num_kv_heads + w.kvh) * p.block_size;
                    const uint32_t off = lane * p.block_size * 128;  // page lane's rows in a 64-column block
                    const uint32_t full = full0 + 8 * stage;
                    if (lane == 0) ok = mbar_wait(empty0 + 8 * stage, phase ^ 1u, p.status, abort_flag);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    if (lane == 0) {
                        if (bytes) mbar_expect_tx(full, bytes);
                        else mbar_arrive(full);
                    }
                    __syncwarp();
                    if (have) {
                        const uint32_t dst = ring + stage * kTileBytes + off;
                        tma_load_2d(dst, map, 0, row, full);
                        tma_load_2d(dst + kBlkBytes, map, 64, row, full);
                    }
                    ++fill;
                    if (++stage == nst) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
        // after an abort, wait (bounded) for this ring's copies still landing
        if (lane == 0 && *abort_flag) {
            const uint64_t t0 = global_timer_ns();
            const uint32_t first = fill > nst ? fill - nst : 0u;
            for (uint32_t f = first; f < fill; ++f)
                while (!mbar_try_wait(full0 + 8 * (f % nst), (f / nst) & 1u))
                    if (global_timer_ns() - t0 > kWaitLimitNs) break;
        }
    } else if (warp == 3) {
        // ----------------------------- query loader -----------------------------
        // an item's 128 query rows (row = token * G + head) as a K-major,
        // 128B-swizzled operand, the layout of a K tile, once the previous
        // item's last QK has released the buffer: two TMA boxes when the
        // item's tokens end inside the batch and inside the map's extent
        // (rows past the sequence then hold the next sequence's queries:
        // every key is masked for them and they are never written out), else
        // 16-byte copies zero-filled past the sequence, handed to the async
        // proxy (also when a sequence before it broke max_seqlen_q and pushed
        // its rows past num_seqs * max_seqlen_q)
        const int64_t total_q = __ldg(p.cu_q + p.num_seqs);
        uint32_t qn = 0;
        bool ok = p.q != nullptr;
        for (int rnd = 0, item; ok && (item = snake_item(rnd, n_items)) >= 0; ++rnd) {
            const Work w = item_work(rnd, item);
            if (w.ntiles == 0) continue;
            if (lane == 0) ok = mbar_wait(q_empty, (qn & 1u) ^ 1u, p.status, abort_flag);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            const int64_t tok0 = static_cast<int64_t>(w.q0) + w.i0;
            const uint32_t dst0 = smem_addr(sQ);
            if (tok0 + p.tq <= total_q && tok0 + p.tq <= p.q_rows) {
                if (lane == 0) {
                    mbar_expect_tx(q_full, kTileBytes);
                    tma_load_3d(dst0, &map_q, 0, w.kvh * p.group, static_cast<int>(tok0), q_full);
                    tma_load_3d(dst0 + kBlkBytes, &map_q, 64, w.kvh * p.group, static_cast<int>(tok0), q_full);
                }
                __syncwarp();
                ++qn;
                continue;
            }
            // (the buffer's previous contents may have come through the async proxy)
            fence_async_smem();
            for (int i = lane; i < kRows * 16; i += 32) {
                const int r = i >> 4, c = i & 15;  // row, 16-byte chunk of the row
                const int t_row = r / p.group, g_row = r - t_row * p.group;
                const bool valid = w.i0 + t_row < w.lq;
                const uint16_t* src =
                    valid ? p.q + ((tok0 + t_row) * p.num_heads + w.kvh * p.group + g_row) * kD + c * 8 : p.q;
                cp_async16(dst0 + (c >> 3) * kBlkBytes + sw128(r, c & 7), src, valid ? 16u : 0u);
            }
            cp_async_wait_all();
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
            ++qn;
        }
        // after an abort, wait (bounded) for a query copy still landing (one
        // at most: each load waits for the buffer's release)
        if (lane == 0 && *abort_flag && qn > 0) {
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(q_full, (qn - 1u) & 1u))
                if (global_timer_ns() - t0 > kWaitLimitNs) break;
        }
    } else if (warp == 1) {
        // -------------------------------- MMA ---------------------------------
        // per item: S[0] = Q K(0)^T, S[1] = Q K(1)^T, then for each tile t:
        // O[c] (+)= P[t&1] V(t) once both softmax warpgroups have written P over S, followed
        // by S[t&1] = Q K(t+2)^T.  One thread waits and issues everything, so the
        // tensor pipe sees each PV before the QK that overwrites its P, and a commit
        // after QK(t+2) also covers PV(t).  The commit after an item's last QK
        // releases the query buffer to the query loader.  (A wait's outcome can
        // differ from lane to lane, and the collectives behind it want every lane:
        // with all lanes waiting and a vote on each wait, the unwindowed prefill
        // took 423 us for 389 and the windowed one 229 for 220.)
        const uint32_t id_qk = mma_idesc(DT == PA_BF16 ? 1 : 0, kRows, kBN, 0);
        const uint32_t id_pv = mma_idesc(DT == PA_BF16 ? 1 : 0, kRows, kD, 1);
        // descriptors are built once; a k-step only adds a constant to the
        // start-address field (bits 0..13, in 16-byte units)
        const uint64_t dk = smem_desc(smem_addr(sK), 16, 1024);
        const uint64_t dv = smem_desc(smem_addr(sV), kBlkBytes, 1024);
        const uint64_t dq = smem_desc(smem_addr(sQ), 16, 1024);
        if (elect_one()) {
            uint32_t k_stage = 0, k_phase = 0;  // K ring position of the next QK
            uint32_t v_stage = 0, v_phase = 0;  // V ring position of the next PV
            uint32_t p_use[2] = {0, 0};         // P[b] handed over so far
            uint32_t pv_count = 0;              // PVs issued so far (all items)
            uint32_t q_cnt = 0;                 // items with tiles
            bool ok = true;
            auto issue_qk = [&](int t, bool last) -> bool {
                if (!mbar_wait(k_full + 8 * k_stage, k_phase, p.status, abort_flag)) return false;
                tc_fence_after();
                const uint32_t b = t & 1;
                const uint64_t dks = dk + k_stage * (kTileBytes >> 4);
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) {
                    // Q and K: 32 bytes per k-step in a 64-column block
                    const uint32_t step = (k / 4) * (kBlkBytes >> 4) + (k % 4) * 2;
                    mma_f16_ss(tmem + kColS + b * kBN, dq + step, dks + step, id_qk, k > 0 ? 1u : 0u);
                }
                mma_commit(s_full + 8 * b);
                mma_commit(k_empty + 8 * k_stage);
                if (last) mma_commit(q_empty);
                if (++k_stage == kStages) {
                    k_stage = 0;
                    k_phase ^= 1u;
                }
                return true;
            };
            // the next item's bookkeeping is done after an item's first QKs, while
            // the softmax warps work on its first tile, not between two items
            int item = snake_item(0, n_items);
            Work w_next{};
            if (item >= 0) w_next = item_work(0, item);
            for (int rnd = 0; ok && item >= 0; ++rnd) {
                const Work w = w_next;
                const int item2 = snake_item(rnd + 1, n_items);
                if (w.ntiles == 0) {
                    item = item2;
                    if (item >= 0) w_next = item_work(rnd + 1, item);
                    continue;
                }
                ok = mbar_wait(q_full, q_cnt & 1u, p.status, abort_flag);
                const uint32_t col_o = tmem + kColO + (q_cnt & 1u) * kD;  // this item's O
                ++q_cnt;
                if (ok) ok = issue_qk(0, w.ntiles == 1);
                if (ok && w.ntiles > 1) ok = issue_qk(1, w.ntiles == 2);
                item = item2;
                if (item >= 0) w_next = item_work(rnd + 1, item);
                for (int t = 0; t < w.ntiles && ok; ++t) {
                    const int y = t & 1;
                    // (V has mostly landed by the time the weights are there: the other way
                    // round the windowed prefill ran 2 % slower)
                    ok = mbar_wait(v_full + 8 * v_stage, v_phase, p.status, abort_flag) &&
                         mbar_wait(p_full + 8 * y, p_use[y] & 1u, p.status, abort_flag);
                    if (!ok) break;
                    ++p_use[y];
                    tc_fence_after();
                    const uint64_t dvs = dv + v_stage * (kTileBytes >> 4);
                    constexpr int kParts = DT == PA_BF16 ? 2 : 1;  // bf16: hi and lo weights
#pragma unroll
                    for (int part = 0; part < kParts; ++part) {
#pragma unroll
                        for (int j = 0; j < kBN / 16; ++j) {
                            // keys 16j..16j+15: P at 8 columns of half j/4 (hi at +0, lo at +32);
                            // V: 2048 bytes per 16 keys
                            mma_f16_ts(col_o, tmem + kColS + y * kBN + (j / 4) * 64 + part * 32 + (j % 4) * 8,
                                       dvs + j * (2048 >> 4), id_pv, (t > 0 || part > 0 || j > 0) ? 1u : 0u);
                        }
                    }
                    mma_commit(v_empty + 8 * v_stage);
                    mma_commit(o_done + 8 * (pv_count & 1u));
                    ++pv_count;
                    if (++v_stage == kStagesV) {
                        v_stage = 0;
                        v_phase ^= 1u;
                    }
                    if (t + 2 < w.ntiles) ok = issue_qk(t + 2, t + 3 == w.ntiles);
                }
            }
            // every MMA issued here is complete before tensor memory is freed
            mma_commit(mma_done);
        }
        __syncwarp();
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(mma_done, 0u))
            if (global_timer_ns() - t0 > kWaitLimitNs) {
                report(p.status, PA_ERR_TIMEOUT);
                break;
            }
    } else if (warp >= kSoftWarp0) {
        // ------------------------------ softmax -------------------------------
        // Both warpgroups work on every key tile: warpgroup x takes keys
        // 64x .. 64x+63 of S[t&1] and the value columns 64x .. 64x+63 of O, row
        // r = its tensor-memory lane.  Both use one reference max m per row.
        // Fast path: weights against the current m, and a barrier that ORs
        // "this row's partial sum left the safe range" over all 256 threads;
        // only then (and on an item's first tile, where m is -inf) do both
        // warpgroups take the tile's true row max, swap it through shared
        // memory, move m, rescale O and recompute.  Between such events the
        // weights may grow up to 2^64 against m (2^15 where they are fp16), inside
        // the range of their type, so no precision is lost.  Every thread of both warpgroups
        // passes the same barriers whatever its waits returned, and stops only
        // on an abort snapshot taken right after the previous barrier.
        // An item's epilogue (O / l out of its O buffer) is deferred to the top
        // of the next item's second key tile (or the end of its first, if it
        // has one): the tensor cores meanwhile run that item's first PV into
        // the other O buffer.
        const int x = (warp - kSoftWarp0) >> 2;   // warpgroup
        const int u = tid - kSoftWarp0 * 32;       // 0..255 over both warpgroups
        const int r = u & 127;                     // row of the tile = tensor-memory lane
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t sbuf = tmem + kColS + 64 * x + lane_base;   // + b * kBN
        const uint32_t tmem_o0 = tmem + kColO + 64 * x + lane_base;  // + c * kD: O[c]
        uint32_t s_use[2] = {0, 0};
        uint32_t n_tiled = 0;  // items with key tiles so far (O[n_tiled & 1] is the current item's)
        uint32_t nbar = 0;     // barriers passed (same count in all 256 threads)
        uint32_t tiles = 0;    // key tiles (= PVs) before the current item
        // partial sums below it need no new max: 2^64, or 2^15 of fp16 weights,
        // which end at 65504 (a sum is at least its largest weight)
        constexpr float kSafe = DT == PA_BF16 ? 18446744073709551616.f : 32768.f;
        // after every barrier among the 256: the abort snapshot of the previous one
        auto snapshot = [&]() -> bool {
            const int stop = snap[(nbar + 1) & 1];
            if (u == 0) snap[nbar & 1] = *abort_flag;
            ++nbar;
            return stop != 0;
        };
        bool stop = false;
        // this row's query row and head in q / out for item w
        auto row_of = [&](const Work& w, bool& valid) -> int64_t {
            const int t_row = r / p.group, g_row = r - t_row * p.group;
            const int qi = w.i0 + t_row;  // query index of this row in its sequence
            valid = qi < w.lq;
            const int qrow = w.q0 + qi;
            const int head = w.kvh * p.group + g_row;
            return (static_cast<int64_t>(qrow) * p.num_heads + head) * kD;
        };
        // the pending epilogue: the previous item with key tiles, not yet
        // written out; its per-thread row offset and partial sum wait in
        // shared memory (pend_off[u], pend_l[u])
        bool pend = false, pend_ok = false;
        // all 256 threads: the pending item's O / l out of O buffer o_col (this
        // thread's columns), its last PV number g; false once an abort
        // snapshot says stop.  These threads saw an S committed after the
        // item's last PV (the next item's first QK) or, when no item follows,
        // after the PV before it (the item's last QK); and the PV two after it
        // needs weights not written yet: the wait neither aliases nor passes early.
        auto finish = [&](uint32_t o_col, uint32_t g) -> bool {
            pend = false;
            bool okf = pend_ok && mbar_wait(o_done + 8 * (g & 1u), (g >> 1) & 1u, p.status, abort_flag);
            okf = __all_sync(0xffffffffu, okf);
            const float my_l = pend_l[u];
            const int64_t my_off = pend_off[u];
            xch[((nbar & 1) * 2 + x) * kRows + r] = my_l;
            named_bar_sync(3, 256);
            if (snapshot()) return false;
            if (okf) {
                tc_fence_after();
                const float L = my_l + xch[((((nbar - 1) & 1) * 2) + (x ^ 1)) * kRows + r];
                const float inv = L > 0.f ? 1.f / L : 0.f;
                uint16_t* dst_e = static_cast<uint16_t*>(p.out) + my_off + 64 * x;
                // 32-byte stores (whole sectors) when out allows them: a row's
                // 16 columns start at a multiple of 32 bytes from out
                const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
                [[maybe_unused]] uint64_t zero = 0ull;  // NaN once an element is not finite
#pragma unroll
                for (int c0 = 0; c0 < 64; c0 += 32) {
                    float o[32];
                    tmem_ld32(o_col + c0, o);
                    if constexpr (WIN) {
#pragma unroll
                        for (int j = 0; j < 32; j += 2) zero = f2fma(f2pack(o[j], o[j + 1]), 0ull, zero);
                    }
                    if (my_off >= 0) {
                        uint32_t wv[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) wv[j] = pack2<DT>(o[2 * j] * inv, o[2 * j + 1] * inv);
                        if (wide) {
#pragma unroll
                            for (int j = 0; j < 2; ++j) st_global_v8(dst_e + c0 + 16 * j, wv + 8 * j);
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                *reinterpret_cast<uint4*>(dst_e + c0 + 8 * j) =
                                    make_uint4(wv[4 * j], wv[4 * j + 1], wv[4 * j + 2], wv[4 * j + 3]);
                        }
                    }
                }
                if constexpr (WIN) {
                    const float2 z = f2unpack(zero);
                    if (my_off >= 0 && !(z.x + z.y == 0.f) && L < INFINITY) *redo = 1;
                }
                // a later item's first PV overwrites this O buffer: its p_full
                // arrival orders that after these reads
                tc_fence_before();
            }
            return true;
        };
        for (int rnd = 0; !stop; ++rnd) {
            // past the last item, one round more writes its O
            const int item = snake_item(rnd, n_items);
            const bool end = item < 0;
            if (end && !pend) break;
            const Work w = end ? Work{} : item_work(rnd, item);
            const int shift = w.lk - w.lq;
            const int t_row = r / p.group;
            const int qi = w.i0 + t_row;  // query index of this row in its sequence
            bool row_valid;
            const int64_t row_off = row_of(w, row_valid);
            // keys [0, lim) visible (window: of these, none from the sinks' end to
            // lo; for the item's rows together, to lo_item)
            const int gone = WIN ? w.skip * p.block_size : 0;
            const int lk = w.lk - gone;
            const int lim = (WIN || p.causal ? min(w.lk, shift + qi + 1) : w.lk) - gone;
            [[maybe_unused]] const int lo = first_key<WIN>(p, shift + qi) - gone;
            [[maybe_unused]] const int lo_item = first_key<WIN>(p, shift + w.i0) - gone;
            uint16_t* dst = static_cast<uint16_t*>(p.out) + row_off + 64 * x;
            if (w.ntiles == 0 && !end) {
                // no visible key for any row of the item: output 0
                if (row_valid) {
                    for (int c = 0; c < 64; c += 8)
                        *reinterpret_cast<uint4*>(dst + c) = make_uint4(0u, 0u, 0u, 0u);
                }
                continue;
            }
            const uint32_t tmem_o = tmem_o0 + (n_tiled & 1u) * kD;  // this item's O
            ++n_tiled;
            float m = -INFINITY, l = 0.f;  // reference max (same in both warpgroups), own partial sum
            bool ok = true;
            const uint64_t sc2 = f2pack(p.scale_log2, p.scale_log2);
            for (int t = 0;; ++t) {
                // the previous item's O is the other buffer; its last PV is
                // the one before this item's first
                if (pend && (t == 1 || end) && !finish(tmem_o0 + (n_tiled & 1u) * kD, tiles - 1)) {
                    stop = true;
                    break;
                }
                if (t >= w.ntiles) break;
                const int b = t & 1;
                const int key0 = t * kBN + 64 * x;  // first key of this thread's 64 columns
                const int vis = row_valid ? lim - key0 : 0;  // visible keys of these columns: [0, vis)
                // ... without [hid0, hid1)
                [[maybe_unused]] const int hid0 = WIN ? max(sinks_of<WIN>(p) - key0, 0) : 0;
                [[maybe_unused]] const int hid1 = WIN ? min(lo - key0, 64) : 0;
                ok = ok && mbar_wait(s_full + 8 * b, s_use[b] & 1u, p.status, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();  // for both reads of S below
                ++s_use[b];
                float e[64];
                float sum = 0.f;
                bool over = false;
                // (window: an item's first tile has no reference, straight to the
                // true maximum)
                const bool first = WIN && t == 0;
                if (ok && !first) {
                    tmem_ld64(sbuf + b * kBN, e);
                    hide_keys<WIN>(e, vis, hid0, hid1);
                    if (m == -INFINITY) {
                        // no reference yet: the slow path, unless these columns
                        // are all masked for this row (weights 0)
                        over = vis > 0 && !(WIN && hid0 == 0 && hid1 >= min(vis, 64));
#pragma unroll
                        for (int i = 0; i < 64; ++i) e[i] = 0.f;
                    } else {
                        // p = 2^(s*scale - m): one packed FFMA per pair and one exp2
                        // per score (masked scores are -inf and give 0)
                        const uint64_t nb2 = f2pack(-m, -m);
#pragma unroll
                        for (int i = 0; i < 64; i += 2) {
                            const float2 a = f2unpack(f2fma(f2pack(e[i], e[i + 1]), sc2, nb2));
                            e[i] = ex2(a.x);
                            e[i + 1] = ex2(a.y);
                        }
                        uint64_t s8[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            s8[j] = f2add(f2add(f2pack(e[2 * j], e[2 * j + 1]), f2pack(e[2 * j + 8], e[2 * j + 9])),
                                          f2add(f2pack(e[2 * j + 16], e[2 * j + 17]), f2pack(e[2 * j + 24], e[2 * j + 25])));
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            s8[j] = f2add(s8[j], f2add(f2add(f2pack(e[2 * j + 32], e[2 * j + 33]), f2pack(e[2 * j + 40], e[2 * j + 41])),
                                                       f2add(f2pack(e[2 * j + 48], e[2 * j + 49]), f2pack(e[2 * j + 56], e[2 * j + 57]))));
                        const float2 s01 = f2unpack(f2add(f2add(s8[0], s8[1]), f2add(s8[2], s8[3])));
                        sum = s01.x + s01.y;
                        over = !(sum < kSafe);  // also catches inf and NaN
                    }
                }
                bool any = true;
                if (!first) {
                    any = bar_red_or(2, 256, over);
                    if (snapshot()) {
                        stop = true;
                        break;
                    }
                }
                if (any) {
                    // slow path (all 256 threads): the tile's true row max over both
                    // halves, a new reference, O and l rescaled, weights recomputed
                    float mx = -INFINITY;
                    if (ok) {
                        tmem_ld64(sbuf + b * kBN, e);
                        hide_keys<WIN>(e, vis, hid0, hid1);
                        float m8[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) m8[j] = fmax3(e[8 * j], e[8 * j + 1], e[8 * j + 2]);
#pragma unroll
                        for (int j = 0; j < 8; ++j) m8[j] = fmax3(m8[j], e[8 * j + 3], e[8 * j + 4]);
#pragma unroll
                        for (int j = 0; j < 8; ++j) m8[j] = fmax3(m8[j], e[8 * j + 5], e[8 * j + 6]);
#pragma unroll
                        for (int j = 0; j < 8; ++j) m8[j] = fmaxf(m8[j], e[8 * j + 7]);
                        mx = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
                    }
                    xch[((nbar & 1) * 2 + x) * kRows + r] = mx;
                    named_bar_sync(3, 256);
                    if (snapshot()) {
                        stop = true;
                        break;
                    }
                    if (!ok) continue;
                    // scale > 0: the max commutes with it
                    mx = fmaxf(mx, xch[((((nbar - 1) & 1) * 2) + (x ^ 1)) * kRows + r]) * p.scale_log2;
                    const bool grow = mx > m;
                    const float a = grow ? ex2(m - mx) : 1.f;  // 0 when m = -inf
                    // O holds PV(0..t-1) against m: rescale it (warp-wide accesses,
                    // factor 1 for other rows) once PV(t-1) is complete.  PV number g
                    // completes a phase of o_done[g & 1]; the previous phase of that
                    // barrier belongs to PV(t-3), complete since it precedes QK(t).
                    if (__any_sync(0xffffffffu, grow) && t > 0) {
                        const uint32_t g = tiles + t - 1;
                        ok = mbar_wait(o_done + 8 * (g & 1u), (g >> 1) & 1u, p.status, abort_flag);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) continue;
                        tc_fence_after();
#pragma unroll
                        for (int c0 = 0; c0 < 64; c0 += 32) {
                            float o[32];
                            tmem_ld32(tmem_o + c0, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= a;
                            tmem_st32(tmem_o + c0, o);
                        }
                    }
                    if (grow) {
                        l *= a;
                        m = mx;
                    }
                    const float nb = m == -INFINITY ? 0.f : -m;
                    const uint64_t nb2 = f2pack(nb, nb);
#pragma unroll
                    for (int i = 0; i < 64; i += 2) {
                        const float2 q2 = f2unpack(f2fma(f2pack(e[i], e[i + 1]), sc2, nb2));
                        e[i] = ex2(q2.x);
                        e[i + 1] = ex2(q2.y);
                    }
                    float r8[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) r8[j] = (e[j] + e[j + 8]) + (e[j + 16] + e[j + 24]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) r8[j] += (e[j + 32] + e[j + 40]) + (e[j + 48] + e[j + 56]);
                    sum = ((r8[0] + r8[1]) + (r8[2] + r8[3])) + ((r8[4] + r8[5]) + (r8[6] + r8[7]));
                }
                if (!ok) continue;
                l += sum;
                // values past Lk in the last tile may hold anything: zero those
                // V rows (after the tile landed) so zero weights never meet NaN;
                // window: also those that no row of the item sees, from the sinks'
                // end to the first row's lo
                const int hole0 = WIN ? max(sinks_of<WIN>(p) - t * kBN, 0) : 0;
                const int hole1 = WIN ? min(lo_item - t * kBN, kBN) : 0;
                if (t * kBN + kBN > lk || (WIN && hole0 < hole1)) {
                    const uint32_t f = tiles + t;
                    ok = mbar_wait(v_full + 8 * (f % kStagesV), (f / kStagesV) & 1u, p.status, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) continue;
                    uint8_t* vt = sV + (f % kStagesV) * kTileBytes;
                    auto zero_rows = [&](int first, int end) {
                        for (int ci = u; ci < (end - first) * 16; ci += 256) {
                            const int rr = first + (ci >> 4), c = ci & 15;
                            *reinterpret_cast<uint4*>(vt + (c >> 3) * kBlkBytes + sw128(rr, c & 7)) =
                                make_uint4(0u, 0u, 0u, 0u);
                        }
                    };
                    zero_rows(max(0, lk - t * kBN), kBN);
                    if constexpr (WIN) zero_rows(hole0, hole1);
                    fence_async_smem();
                }
                // P over S in tensor memory as 16-bit pairs (bf16: hi at columns
                // 0..31 of this warpgroup's 64 and the remainder lo at 32..63, both
                // truncated, ~16 bits together)
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // keys 32h .. 32h+31 = columns 16h .. 16h+15
                    uint32_t hw[16], lw[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float a = e[32 * h + 2 * j], c = e[32 * h + 2 * j + 1];
                        if constexpr (DT == PA_BF16) {
                            hw[j] = hi_halves(a, c);
                            const float2 lo = f2unpack(f2add(f2pack(a, c), f2pack(-__uint_as_float(hw[j] << 16),
                                                                                -__uint_as_float(hw[j] & 0xffff0000u))));
                            lw[j] = hi_halves(lo.x, lo.y);
                        } else {
                            hw[j] = pack2<DT>(a, c);
                        }
                    }
                    tmem_st16(sbuf + b * kBN + 16 * h, hw);
                    if constexpr (DT == PA_BF16) tmem_st16(sbuf + b * kBN + 32 + 16 * h, lw);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * b);
            }
            if (stop || end) break;
            tiles += w.ntiles;
            pend = true;
            pend_ok = ok;
            pend_l[u] = l;
            pend_off[u] = row_valid ? row_off : -1;
        }
    }
    // ---- teardown: every role is done; free tensor memory ----
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
    if constexpr (WIN) {
        // (every copy has landed and been used: the K ring's memory is free)
        if (*redo && !*abort_flag) redo_rows<DT>(p, prefix, order, n_items, reinterpret_cast<float*>(sK) + warp * kD);
    }
}

// packed K or V as a 3-D tensor {head_size, num_kv_heads, total rows}; a box
// is 64 elements x 1 head x 128 rows
bool make_packed_map(CUtensorMap* map, const void* base, int64_t total_k, int num_kv_heads, int dtype) {
    const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(num_kv_heads),
                                static_cast<cuuint64_t>(total_k)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kD) * 2,
                                   static_cast<cuuint64_t>(num_kv_heads) * kD * 2};
    const cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(kBN)};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(map, dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                          3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// Token extent of the query map: num_seqs * max_seqlen_q, a bound on the real count
// (which only the device knows): boxes are loaded only for items whose tokens end before
// the real count and inside this extent, so no copy reaches past the real rows.
int32_t q_map_rows(int num_seqs, int max_q) {
    const int64_t bound = static_cast<int64_t>(num_seqs) * max_q;
    return static_cast<int32_t>(bound < INT32_MAX ? bound : INT32_MAX);
}

// launch shared by the paged and packed entry points (p filled in, maps built)
template <bool PACKED, bool WIN>
pa_status launch_prefill(const ParamsOf<WIN>& p, pa_dtype dtype, const CUtensorMap& map_k,
                         const CUtensorMap& map_v, const CUtensorMap& map_q, pa_stream_t stream) {
    // shared memory past the fixed layout: the tile prefix (B+1 ints), the
    // work order (up to every query tile the bounds allow, within what the
    // device offers) and the sort's [12 warps][64 classes] counts
    const int base = kSmemBytes + (p.num_seqs + 1) * 4 + 1024;
    if (base > device_max_smem_optin()) return PA_ERR_UNSUPPORTED;
    const int64_t tiles_bound = static_cast<int64_t>(p.num_seqs) * ((p.max_q + p.tq - 1) / p.tq);
    // (2 KB kept back for the kernel's static shared memory)
    const int64_t room = (device_max_smem_optin() - 2048 - base) / 4 - (kThreads / 32) * 64;
    ParamsOf<WIN> q = p;
    q.order_cap = static_cast<int32_t>(room <= 0 ? 0 : (tiles_bound < room ? tiles_bound : room));
    const int smem = base + (q.order_cap > 0 ? (q.order_cap + (kThreads / 32) * 64) * 4 : 0);
    static LaunchCache cache_bf16, cache_f16;
    auto kern = dtype == PA_BF16 ? paged_prefill_tc_kernel<PA_BF16, PACKED, WIN>
                                : paged_prefill_tc_kernel<PA_F16, PACKED, WIN>;
    const int per_sm = blocks_per_sm(kern, kThreads, smem, dtype == PA_BF16 ? cache_bf16 : cache_f16);
    if (per_sm <= 0) return PA_ERR_CUDA;
    const int64_t max_items =
        static_cast<int64_t>(p.num_seqs) * ((p.max_q + p.tq - 1) / p.tq) * p.num_kv_heads;
    const int64_t cap = static_cast<int64_t>(device_sm_count()) * per_sm;
    const int grid = static_cast<int>(max_items < cap ? max_items : cap);
    if (grid <= 0) return PA_OK;
    return launch_pdl(kern, grid, kThreads, smem, reinterpret_cast<cudaStream_t>(stream), map_k, map_v, map_q, q) ==
                   cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // namespace
}  // namespace pa

using namespace pa;

namespace pa {
namespace {

// pa_prefill_varlen, and pa_prefill_varlen_window when window > 0; no_copies: the
// test hook's launch
pa_status prefill_entry(void* out, const void* q, pa_dtype q_dtype, const pa_kv_cache* cache,
                        const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* cu_seq_lens_q,
                        const int32_t* cu_seq_lens_k, int32_t num_seqs, int32_t max_seqlen_q, int32_t max_seqlen_k,
                        int32_t num_heads, float scale, int32_t causal, int32_t window, int32_t sinks,
                        int32_t* dev_status, pa_stream_t stream, bool no_copies = false) {
    pa_status st = check_cache(cache);
    if (st != PA_OK) return st;
    if (num_seqs < 0 || num_heads <= 0 || max_blocks_per_seq <= 0 || max_seqlen_q < 0 ||
        max_seqlen_k < 0 || !(scale == scale))
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || max_seqlen_q == 0) return PA_OK;
    if (out == nullptr || q == nullptr || block_table == nullptr || cu_seq_lens_q == nullptr ||
        cu_seq_lens_k == nullptr)
        return PA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(out) & 15u) || (reinterpret_cast<uintptr_t>(q) & 15u))
        return PA_ERR_INVALID_ARG;
    if (num_heads % cache->num_kv_heads != 0) return PA_ERR_INVALID_ARG;
    const int group = num_heads / cache->num_kv_heads;
    if (cache->head_size != kD) return PA_ERR_UNSUPPORTED;
    if (group != 1 && group != 2 && group != 4 && group != 8) return PA_ERR_UNSUPPORTED;
    if (q_dtype != PA_F16 && q_dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (cache->kv_dtype != q_dtype) return PA_ERR_UNSUPPORTED;
    const int bs = cache->block_size;
    if (bs != 16 && bs != 32 && bs != 64) return PA_ERR_UNSUPPORTED;
    if (num_seqs > kMaxSeqs) return PA_ERR_UNSUPPORTED;
    const int64_t rows = cache->num_blocks * cache->num_kv_heads * bs;
    if (rows > INT32_MAX) return PA_ERR_UNSUPPORTED;

    PrefillParams p{};
    p.out = out;
    p.q = static_cast<const uint16_t*>(q);
    p.block_table = block_table;
    p.cu_q = cu_seq_lens_q;
    p.cu_k = cu_seq_lens_k;
    p.status = dev_status;
    p.num_blocks = cache->num_blocks;
    p.block_size = bs;
    p.num_kv_heads = cache->num_kv_heads;
    p.num_heads = num_heads;
    p.group = group;
    p.tq = kRows / group;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.max_q = max_seqlen_q;
    p.max_k = max_seqlen_k;
    p.causal = causal ? 1 : 0;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.total_k = -1;

    CUtensorMap map_k, map_v;
    if (!make_cache_map(&map_k, cache->k_cache, rows, q_dtype, bs) ||
        !make_cache_map(&map_v, cache->v_cache, rows, q_dtype, bs))
        return PA_ERR_CUDA;
    CUtensorMap map_q;
    if (!make_q_map(&map_q, q, num_heads, group, q_map_rows(num_seqs, max_seqlen_q), q_dtype)) return PA_ERR_CUDA;
    p.q_rows = q_map_rows(num_seqs, max_seqlen_q);
    if (no_copies) p.q = nullptr;
    if (window > 0) {
        // (a window, or sinks, past the longest sequence change nothing more)
        const int32_t most = max_seqlen_k > 1 ? max_seqlen_k : 1;
        WindowParams w{p, window < most ? window : most, sinks < most ? sinks : most, 0,
                       static_cast<const uint16_t*>(cache->k_cache), static_cast<const uint16_t*>(cache->v_cache)};
        w.head = (w.sinks + bs - 1) / bs;
        return launch_prefill<false, true>(w, q_dtype, map_k, map_v, map_q, stream);
    }
    return launch_prefill<false, false>(p, q_dtype, map_k, map_v, map_q, stream);
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_prefill_varlen(void* out, const void* q, pa_dtype q_dtype,
                                       const pa_kv_cache* cache, const int32_t* block_table,
                                       int32_t max_blocks_per_seq, const int32_t* cu_seq_lens_q,
                                       const int32_t* cu_seq_lens_k, int32_t num_seqs,
                                       int32_t max_seqlen_q, int32_t max_seqlen_k, int32_t num_heads,
                                       float scale, int32_t causal, int32_t* dev_status,
                                       pa_stream_t stream) {
    return pa::prefill_entry(out, q, q_dtype, cache, block_table, max_blocks_per_seq, cu_seq_lens_q, cu_seq_lens_k,
                             num_seqs, max_seqlen_q, max_seqlen_k, num_heads, scale, causal, 0, 0, dev_status, stream);
}

extern "C" pa_status pa_prefill_varlen_window(void* out, const void* q, pa_dtype q_dtype, const pa_kv_cache* cache,
                                              const int32_t* block_table, int32_t max_blocks_per_seq,
                                              const int32_t* cu_seq_lens_q, const int32_t* cu_seq_lens_k,
                                              int32_t num_seqs, int32_t max_seqlen_q, int32_t max_seqlen_k,
                                              int32_t num_heads, float scale, int32_t window, int32_t num_sinks,
                                              int32_t* dev_status, pa_stream_t stream) {
    if (window <= 0 || num_sinks < 0) return PA_ERR_INVALID_ARG;
    // (the running maximum is taken over unscaled scores)
    if (!(scale > 0.f) || !std::isfinite(scale)) return PA_ERR_INVALID_ARG;
    return pa::prefill_entry(out, q, q_dtype, cache, block_table, max_blocks_per_seq, cu_seq_lens_q, cu_seq_lens_k,
                             num_seqs, max_seqlen_q, max_seqlen_k, num_heads, scale, 1, window, num_sinks, dev_status,
                             stream);
}

extern "C" pa_status pa_prefill_test_wait_timeout(void* out, const void* q, pa_dtype q_dtype, const pa_kv_cache* cache,
                                                  const int32_t* block_table, int32_t max_blocks_per_seq,
                                                  const int32_t* cu_seq_lens_q, const int32_t* cu_seq_lens_k,
                                                  int32_t num_seqs, int32_t max_seqlen_q, int32_t max_seqlen_k,
                                                  int32_t num_heads, float scale, int32_t window, int32_t num_sinks,
                                                  int32_t* dev_status, pa_stream_t stream) {
    if (window < 0 || num_sinks < 0 || !(scale > 0.f) || !std::isfinite(scale)) return PA_ERR_INVALID_ARG;
    return pa::prefill_entry(out, q, q_dtype, cache, block_table, max_blocks_per_seq, cu_seq_lens_q, cu_seq_lens_k,
                             num_seqs, max_seqlen_q, max_seqlen_k, num_heads, scale, 1, window, num_sinks, dev_status,
                             stream, true);
}

extern "C" pa_status pa_prefill_varlen_packed(void* out, const void* q, const void* k, const void* v,
                                              pa_dtype dtype, const int32_t* cu_seq_lens_q,
                                              const int32_t* cu_seq_lens_k, int32_t num_seqs,
                                              int32_t max_seqlen_q, int32_t max_seqlen_k, int64_t total_k,
                                              int32_t num_heads, int32_t num_kv_heads, int32_t head_size,
                                              float scale, int32_t causal, int32_t* dev_status,
                                              pa_stream_t stream) {
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || max_seqlen_q < 0 || max_seqlen_k < 0 ||
        total_k < 0 || !(scale == scale))
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || max_seqlen_q == 0) return PA_OK;
    if (out == nullptr || q == nullptr || cu_seq_lens_q == nullptr || cu_seq_lens_k == nullptr)
        return PA_ERR_INVALID_ARG;
    if (total_k > 0 && (k == nullptr || v == nullptr)) return PA_ERR_INVALID_ARG;
    for (const void* ptr : {static_cast<const void*>(out), q, k, v})
        if (reinterpret_cast<uintptr_t>(ptr) & 15u) return PA_ERR_INVALID_ARG;
    if (num_heads % num_kv_heads != 0) return PA_ERR_INVALID_ARG;
    const int group = num_heads / num_kv_heads;
    if (head_size != kD) return PA_ERR_UNSUPPORTED;
    if (group != 1 && group != 2 && group != 4 && group != 8) return PA_ERR_UNSUPPORTED;
    if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (num_seqs > kMaxSeqs) return PA_ERR_UNSUPPORTED;
    if (total_k > INT32_MAX - kBN) return PA_ERR_UNSUPPORTED;

    PrefillParams p{};
    p.out = out;
    p.q = static_cast<const uint16_t*>(q);
    p.cu_q = cu_seq_lens_q;
    p.cu_k = cu_seq_lens_k;
    p.status = dev_status;
    p.block_size = kBN;
    p.num_kv_heads = num_kv_heads;
    p.num_heads = num_heads;
    p.group = group;
    p.tq = kRows / group;
    p.num_seqs = num_seqs;
    p.max_q = max_seqlen_q;
    p.max_k = max_seqlen_k;
    p.causal = causal ? 1 : 0;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.total_k = total_k;

    // an empty K/V still needs a valid map: point it at q (never read, every
    // sequence then has no key)
    const int64_t rows = total_k > 0 ? total_k : 1;
    CUtensorMap map_k, map_v;
    if (!make_packed_map(&map_k, total_k > 0 ? k : q, rows, num_kv_heads, dtype) ||
        !make_packed_map(&map_v, total_k > 0 ? v : q, rows, num_kv_heads, dtype))
        return PA_ERR_CUDA;
    CUtensorMap map_q;
    if (!make_q_map(&map_q, q, num_heads, group, q_map_rows(num_seqs, max_seqlen_q), dtype)) return PA_ERR_CUDA;
    p.q_rows = q_map_rows(num_seqs, max_seqlen_q);
    return launch_prefill<true, false>(p, dtype, map_k, map_v, map_q, stream);
}
