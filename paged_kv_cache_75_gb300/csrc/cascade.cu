// Varlen attention of groups of sequences that share a prefix, the prefix computed once
// for a group (pa_varlen_cascade), on the 5th-generation tensor cores.
//
// "Как работает paged attention? (детально)" 3.3 and 7: sequences of one prompt (beams,
// samples) and requests with the same prefix refer to the same physical blocks.  What it
// computes is the causal varlen attention of "Paged 어텐션" (Varlen 경로) with the
// softmax taken in parts: over the group's shared blocks its members' query rows, which
// stand side by side in q, fill the 128 rows of a tile whatever member they are of (every
// query sees every shared key, so there is no mask), and each member's own keys follow
// with its causal mask.  A part of keys [a, b) leaves for each row
//     o = sum_j 2^(s_j - m) v_j / l,   lse = m + log2 l,   l = sum_j 2^(s_j - m)
// (s in units of log2), and the merge kernel forms sum_p 2^(lse_p - M) o_p / sum_p 2^(lse_p - M).
//
// The keys of a part stream through the same pipeline as in the prefill: two loader warps
// (K and V rings, TMA through the block table), one query loader, one thread that issues
// every MMA, two softmax warpgroups that split the 128 key columns of a tile.  Work is a
// list of segments (a group's prefix, a sequence's own keys), each of query tiles and parts
// of `part` keys; an entry of it is num_kv_heads items.  Entries are sorted by their key
// tiles, most first, and dealt to the persistent blocks in snake order (tiles that share keys
// then run side by side; one line of work cut into equal runs was even, but read a prefix
// of 65536 tokens once per query tile, 250 us for 190).  Every wait is bounded.
//
// Bound by the softmax warps' chain of 1.1 (fp16) to 1.3 us (bf16) a key tile, 128 rows in
// use or 8; a key tile of bf16 is 0.81 us of tensor work.  On one GB300: 32 questions of 4 to 32
// tokens to 16384 tokens (32/8 heads, bf16) 188 us, tensor pipe 62 %; 64 answers behind 65536
// tokens (64/8, fp16) 132; 32 groups of eight beams behind 256 to 8192 tokens 73, 52 % of DRAM;
// 20 chunks of up to 1024 tokens behind 1024 to 8192 (not stacked) 815, tensor pipe 69 %.
#include <cmath>

#include "decode_launch.cuh"
#include "tcgen05.cuh"

namespace pa {
namespace {

constexpr int kStages = 3;           // depth of the K ring
constexpr int kStagesV = 2;          // depth of the V ring
constexpr int kThreads = 384;        // 12 warps
constexpr int kSoftWarp0 = 4;        // softmax warpgroups = warps 4..7 and 8..11
constexpr uint32_t kTmemCols = 512;
// tensor-memory columns: S[b] (scores of the key tiles t with t & 1 = b, later overwritten
// by the 16-bit weights P) and O[c] (accumulators of the items with key tiles, c = their
// count & 1: one item's O is written out while the next item's first PV goes to the other)
constexpr uint32_t kColS = 0;    // S[b] at b * kBN
constexpr uint32_t kColO = 256;  // O[c] at kColO + c * kD

// shared memory layout (bytes from the 1 KB-aligned base)
constexpr int kOffK = 0;                                // K ring
constexpr int kOffV = kOffK + kStages * kTileBytes;     // V ring
constexpr int kOffQ = kOffV + kStagesV * kTileBytes;    // the item's 128 query rows, laid out like a K tile
constexpr int kOffBar = kOffQ + kTileBytes;
constexpr int kNumBars = 2 * kStages + 2 * kStagesV + 3 * 2 + 3;
constexpr int kOffMisc = kOffBar + kNumBars * 8;
constexpr int kOffXch = kOffMisc + 64;                  // [2 slots][2 warpgroups][128 rows] floats
constexpr int kOffPend = kOffXch + 2 * 2 * kRows * 4;   // [256] int64 destinations, [256] sums, [256] references
constexpr int kItemCache = 64;                          // a CTA's first items, worked out once
constexpr int kOffItems = kOffPend + 256 * 16;          // [kItemCache] Work
constexpr int kSmemBytes = kOffItems + kItemCache * 32;
static_assert(kOffMisc % 8 == 0 && kOffPend % 8 == 0 && kOffItems % 8 == 0 && kSmemBytes % 4 == 0, "alignment");
constexpr int kMaxSegments = 6144;  // num_seqs + num_groups (the prefix array in shared memory)

// A K or V tile in shared memory: groups of eight keys, 2 KB each, of which the first 1 KB
// holds the columns 0 .. 63 (128-byte rows, swizzled) and the second 64 .. 127.  So a whole
// page is one box of a 4-D view of the cache, {64 columns, 8 keys, 2 halves, groups}: with a
// box for each half, a tile's TMA instructions (32 at block size 16) bounded the loads.
constexpr int kGroupBytes = 2048;
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* map, int group, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(bar)
        : "memory");
}
inline bool make_page_map(CUtensorMap* map, const void* base, int64_t rows, int dtype, int block_size) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[4] = {64, 8, 2, static_cast<cuuint64_t>(rows / 8)};
    const cuuint64_t strides[3] = {kD * 2, 128, 8 * kD * 2};
    const cuuint32_t box[4] = {64, 8, 2, static_cast<cuuint32_t>(block_size / 8)};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = fn(map, dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                          4, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

struct CascadeParams {
    void* out;
    const uint16_t* q;  // NULL (pa_varlen_cascade_test_wait_timeout): no copy is issued, every wait runs out
    const int32_t* block_table;
    const int32_t* cu_q;
    const int32_t* cu_k;
    const int32_t* cu_groups;
    const int32_t* shared_lens;
    float* ws_lse;  // [total_q * num_heads][max_parts]
    float* ws_o;    // [total_q * num_heads][max_parts][kD]
    int32_t* status;
    int64_t num_blocks;
    int32_t block_size;
    int32_t num_kv_heads;
    int32_t num_heads;
    int32_t group;  // num_heads / num_kv_heads
    int32_t tq;     // query tokens per tile (128 / group)
    int32_t num_seqs;
    int32_t num_groups;
    int32_t max_blocks;
    int32_t max_q;
    int32_t max_k;
    int32_t max_group;
    int32_t max_shared;
    int32_t total_q;
    int32_t part;       // keys of a part (a multiple of kBN)
    int32_t tail_from;  // a prefix's query tiles from this one on
    int32_t tail_part;  // have parts of so many keys instead
    int32_t max_parts;
    int32_t own;        // the sequences' own keys too, or the prefixes alone
    int32_t stack;      // groups share; 0: every sequence's keys are one segment
    int32_t own_base;   // behind a prefix, the own keys' parts are numbered from here
    // own = 0: these parts, of own_part keys, are the decode kernel's, which takes the
    // sequences' lengths from ws_lens

    int32_t own_part;
    int32_t* ws_lens;
    int32_t order_cap;  // entries the shared-memory work order holds (set by the launch)
    float scale_log2;   // scale * log2(e)
};

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b > 0); }

// lengths of sequence b; false if they break the stated bounds
__device__ __forceinline__ bool seq_lens_ok(const CascadeParams& p, int b, int& q0, int& lq, int& lk) {
    q0 = __ldg(p.cu_q + b);
    const int q1 = __ldg(p.cu_q + b + 1), k0 = __ldg(p.cu_k + b), k1 = __ldg(p.cu_k + b + 1);
    lq = q1 - q0;
    lk = k1 - k0;
    return q0 >= 0 && q1 >= q0 && q1 <= p.total_q && k0 >= 0 && k1 >= k0 && lq <= p.max_q && lk <= p.max_k &&
           static_cast<int64_t>(lk) <= static_cast<int64_t>(p.max_blocks) * p.block_size;
}

struct Group {
    int b0, b1, s0;
    bool ok;      // within the stated bounds
    bool shares;  // its prefix is a segment of its own
};
__device__ __forceinline__ Group group_at(const CascadeParams& p, int g) {
    Group r;
    r.b0 = __ldg(p.cu_groups + g);
    r.b1 = __ldg(p.cu_groups + g + 1);
    r.s0 = __ldg(p.shared_lens + g);
    r.ok = r.b0 >= 0 && r.b1 >= r.b0 && r.b1 <= p.num_seqs && r.b1 - r.b0 <= p.max_group && r.s0 >= 0 &&
           r.s0 <= p.max_shared && r.s0 % p.block_size == 0 &&
           static_cast<int64_t>(r.s0) <= static_cast<int64_t>(p.max_blocks) * p.block_size;
    // (a group of one: its prefix and its own keys are one segment)
    r.shares = r.ok && p.stack && r.s0 > 0 && (r.b1 - r.b0 > 1 || !p.own);
    return r;
}
// the group of sequence b (the last whose first sequence is not behind it)
__device__ __forceinline__ Group group_of_seq(const CascadeParams& p, int b) {
    int lo = 0, hi = p.num_groups - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(p.cu_groups + mid) <= b) lo = mid;
        else hi = mid - 1;
    }
    Group g = group_at(p, lo);
    if (b < g.b0 || b >= g.b1) g.ok = g.shares = false;
    return g;
}

// Segments 0 .. num_groups-1 are the groups' prefixes, num_groups + b the own keys of
// sequence b: `tiles` query tiles by `parts` parts of the keys.
struct Segment {
    int tab;          // block-table row
    int q0, nq;       // its query rows
    int start, len;   // its keys: positions start .. start + len - 1
    int shift;        // query row i sees the first shift + i + 1 of them
    int tiles, parts; // (of a prefix's tiles from tail_from on: tail_parts)
    int tail_parts;
    int part0;        // its first part's number, -1: its rows have this part alone
};
constexpr int kNoMask = 1 << 30;
__device__ __forceinline__ Segment segment(const CascadeParams& p, int s, bool check) {
    Segment r{};
    if (s < p.num_groups) {
        const Group g = group_at(p, s);
        if (check && !g.ok) report(p.status, PA_ERR_INVALID_ARG);
        if (check && (s == 0 ? g.b0 != 0 : false)) report(p.status, PA_ERR_INVALID_ARG);
        if (check && s == p.num_groups - 1 && g.b1 != p.num_seqs) report(p.status, PA_ERR_INVALID_ARG);
        if (!g.shares) return r;
        r.tab = g.b0;
        r.q0 = __ldg(p.cu_q + g.b0);
        r.nq = __ldg(p.cu_q + g.b1) - r.q0;
        if (r.q0 < 0 || r.nq <= 0 || r.q0 + static_cast<int64_t>(r.nq) > p.total_q) return Segment{};
        r.len = g.s0;
        r.shift = kNoMask;
        r.tiles = ceil_div(r.nq, p.tq);
        r.parts = ceil_div(g.s0, p.part);
        r.tail_parts = ceil_div(g.s0, p.tail_part);
        return r;
    }
    const int b = s - p.num_groups;
    int lq, lk;
    const bool ok = seq_lens_ok(p, b, r.q0, lq, lk);
    const Group g = group_of_seq(p, b);
    // every query comes after the shared tokens
    const bool fits = g.ok && (lq <= 0 || g.s0 <= lk - lq);
    if (check && (!ok || !fits)) report(p.status, PA_ERR_INVALID_ARG);
    if (!ok || !fits || lq == 0) return Segment{};
    r.tab = b;
    r.nq = lq;
    r.start = g.shares ? g.s0 : 0;
    r.len = lk - r.start;
    r.shift = r.len - lq;
    r.tiles = ceil_div(lq, p.tq);
    r.parts = r.len <= p.part ? 1 : ceil_div(r.len, p.part);
    r.part0 = r.start > 0 ? p.own_base : r.parts > 1 ? 0 : -1;
    return r;
}

// entries of a segment
__device__ __forceinline__ int entries(const CascadeParams& p, const Segment& g) {
    const int tail = g.shift == kNoMask ? max(0, g.tiles - p.tail_from) : 0;
    return (g.tiles - tail) * g.parts + tail * g.tail_parts;
}

struct Work {
    int tab, entry0;  // block-table row, its first entry
    int tok0, ntok;   // query rows
    int kvh;
    int nkeys;        // keys that any of the rows sees; row t sees the first shift + t + 1 of them
    int shift;
    int part;         // the part's number, -1: straight to out
    __device__ __forceinline__ int tiles() const { return nkeys > 0 ? (nkeys + kBN - 1) / kBN : 0; }
};
static_assert(sizeof(Work) == 32, "the item cache holds 32-byte entries");

__device__ __forceinline__ Work entry_work(const CascadeParams& p, const int32_t* prefix, int n_seg, int entry) {
    int lo = 0, hi = n_seg - 1;  // largest s with prefix[s] <= entry
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= entry) lo = mid;
        else hi = mid - 1;
    }
    const Segment g = segment(p, lo, false);
    int e = entry - prefix[lo], tile = 0, parts = max(g.parts, 1), size = p.part;
    if (g.shift == kNoMask && e >= p.tail_from * static_cast<int64_t>(parts)) {
        e -= p.tail_from * parts;
        tile = p.tail_from;
        parts = max(g.tail_parts, 1);
        size = p.tail_part;
    }
    const int part = e % parts;
    tile += e / parts;
    Work w;
    const int i0 = tile * p.tq, k0 = part * size;
    w.tab = g.tab;
    w.entry0 = (g.start + k0) / p.block_size;
    w.tok0 = g.q0 + i0;
    w.ntok = min(p.tq, g.nq - i0);
    w.kvh = 0;
    w.shift = g.shift == kNoMask ? kNoMask : g.shift + i0 - k0;
    w.nkeys = min(min(size, g.len - k0), w.shift + w.ntok);
    w.part = g.part0 < 0 ? -1 : g.part0 + part;
    return w;
}

__device__ __forceinline__ Work work_item(const CascadeParams& p, const int32_t* prefix, int n_seg, const int32_t* order,
                                          int item) {
    int entry = item / p.num_kv_heads;
    const int kvh = item - entry * p.num_kv_heads;
    if (order != nullptr) entry = order[entry];
    Work w = entry_work(p, prefix, n_seg, entry);
    w.kvh = kvh;
    return w;
}

// Stable counting sort of the n entries by their key tiles (64 classes, most first):
// each warp counts a contiguous chunk (lanes of equal class found by match.any), warp 0
// turns the [warp][class] counts into class-major offsets, each warp then places its
// chunk in order.  All threads of the block take part; hist holds 12*64 ints.
__device__ __forceinline__ int entry_class(const CascadeParams& p, const int32_t* prefix, int n_seg, int entry) {
    const int most = max(p.part, p.tail_part) / kBN;
    const int n = min(most, entry_work(p, prefix, n_seg, entry).tiles());
    return 63 - static_cast<int>((static_cast<int64_t>(n) * 64) / (most + 1));  // 0 = most key tiles
}
__device__ void build_order(const CascadeParams& p, const int32_t* prefix, int n_seg, int n, int32_t* order,
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
        const int key = t < t1 ? entry_class(p, prefix, n_seg, t) : 64;
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
        const int key = t < t1 ? entry_class(p, prefix, n_seg, t) : 64;
        const unsigned same = __match_any_sync(0xffffffffu, key);
        if (t < t1) order[h[key] + __popc(same & ((1u << lane) - 1u))] = t;
        __syncwarp();
        if (t < t1 && lane == __ffs(same) - 1) h[key] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
}

// scores of the keys that a row does not see: those from vis on
__device__ __forceinline__ void hide_keys(float (&e)[64], int vis) {
    if (vis < 64) {
#pragma unroll
        for (int i = 0; i < 64; ++i)
            if (i >= vis) e[i] = -INFINITY;
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 1)
cascade_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
               const __grid_constant__ CUtensorMap map_q, const CascadeParams p) {
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
    float* xch = reinterpret_cast<float*>(smem + kOffXch);
    // pending epilogue, per thread: where it goes (row_of), the partial row sum, the reference
    int64_t* pend_off = reinterpret_cast<int64_t*>(smem + kOffPend);
    float* pend_l = reinterpret_cast<float*>(smem + kOffPend + 256 * 8);
    float* pend_m = pend_l + 256;
    int32_t* prefix = reinterpret_cast<int32_t*>(smem + kSmemBytes);  // segments + 1 ints past the fixed layout
    __shared__ int32_t scan_scratch[kThreads / 32];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n_seg = p.num_groups + (p.own ? p.num_seqs : 0);

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
        snap[0] = 0;
        snap[1] = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }

    // ---- prefix of the segments' entries ----
    {
        const int chunk = (n_seg + kThreads - 1) / kThreads;
        const int s0 = tid * chunk, s1 = min(n_seg, s0 + chunk);
        int local = 0;
        for (int s = s0; s < s1; ++s) {
            const Segment g = segment(p, s, true);
            prefix[s] = local;
            local += entries(p, g);
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
        int before = v - local;
        for (int w = 0; w < warp; ++w) before += scan_scratch[w];
        for (int s = s0; s < s1; ++s) prefix[s] += before;
        if (tid == kThreads - 1) prefix[n_seg] = before + local;
        __syncthreads();
    }
    // ---- work order of the entries (none where every item has a block of its own) ----
    const int n_entries = prefix[n_seg];
    const int32_t* order = nullptr;
    if (n_entries <= p.order_cap && static_cast<int64_t>(n_entries) * p.num_kv_heads > gridDim.x) {
        int32_t* ord = prefix + n_seg + 1;
        build_order(p, prefix, n_seg, n_entries, ord, ord + p.order_cap);
        order = ord;
    }
    // what the decode kernel goes by: a sequence's length, or its shared length where it
    // has no query (no keys of its own)
    if (!p.own && blockIdx.x == 0) {
        for (int b = tid; b < p.num_seqs; b += kThreads) {
            int q0, lq, lk;
            const bool ok = seq_lens_ok(p, b, q0, lq, lk);
            const Group g = group_of_seq(p, b);
            const bool good = ok && g.ok && (lq == 0 || (g.s0 <= lk - lq && q0 == b));
            if (!good) report(p.status, PA_ERR_INVALID_ARG);
            p.ws_lens[b] = good && lq == 1 ? lk : g.ok ? g.s0 : 0;
        }
    }
    const uint32_t tmem = uniform(*tmem_slot);
    const int n_items = n_entries * p.num_kv_heads;
    // this CTA's first kItemCache items, worked out once: every role's item
    // loop reads them from here (item_work) instead of searching the tile
    // prefix and reading the sequence lengths at each item boundary
    Work* item_cache = reinterpret_cast<Work*>(smem + kOffItems);
    if (tid < kItemCache) {
        const int item = snake_item(tid, n_items);
        if (item >= 0) item_cache[tid] = work_item(p, prefix, n_seg, order, item);
    }
    __syncthreads();
    auto item_work = [&](int rnd, int item) -> Work {
        return rnd < kItemCache ? item_cache[rnd] : work_item(p, prefix, n_seg, order, item);
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
        {
            const int ppt = kBN / p.block_size;  // pages per tile (2, 4 or 8)
            for (int rnd = 0, item; ok && (item = snake_item(rnd, n_items)) >= 0; ++rnd) {
                const Work w = item_work(rnd, item);
                const int32_t* bt_row = p.block_table + static_cast<int64_t>(w.tab) * p.max_blocks + w.entry0;
                // Page ids come in batches of four tiles (a lane each, -1: past the keys,
                // -2: bad id), the next batch's ahead of time
                const int ntiles = w.tiles();
                const int pages = (w.nkeys + p.block_size - 1) / p.block_size;
                auto ids_from = [&](int pg0) -> int32_t {
                    const int pg = pg0 + lane;
                    if (lane >= 4 * ppt || pg >= pages) return -1;
                    const int32_t x = __ldg(bt_row + pg);
                    if (x >= 0 && x < p.num_blocks) return x;
                    // both loader warps read the id; one reports it
                    if (kv == 0) report(p.status, PA_ERR_BAD_BLOCK);
                    return -2;
                };
                int32_t id = -1, id_next = ntiles > 0 ? ids_from(0) : -1;
                for (int t = 0; t < ntiles && ok; ++t) {
                    if ((t & 3) == 0) {
                        id = id_next;
                        id_next = t + 4 < ntiles ? ids_from((t + 4) * ppt) : -1;
                    }
                    // lane k < ppt holds the id of page k of this tile
                    const int from = (t & 3) * ppt + (lane & 7);
                    const int my_id = __shfl_sync(0xffffffffu, id, from & 31);
                    const bool have = lane < ppt && my_id >= 0;
                    const uint32_t bytes =
                        static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, have))) * 2u * p.block_size * kD;
                    const int group = (my_id * p.num_kv_heads + w.kvh) * (p.block_size / 8);
                    const uint32_t full = full0 + 8 * stage;
                    if (lane == 0) ok = mbar_wait(empty0 + 8 * stage, phase ^ 1u, p.status, abort_flag);
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    if (lane == 0) {
                        if (bytes) mbar_expect_tx(full, bytes);
                        else mbar_arrive(full);
                    }
                    __syncwarp();
                    if (have) tma_load_page(ring + stage * kTileBytes + lane * p.block_size * (kD * 2), map, group, full);
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
        // 128B-swizzled operand, the layout of a K tile, once the previous item's
        // last QK has released the buffer: two TMA boxes when the tile ends inside q
        // (rows past the item's tokens then hold other queries: every key is masked
        // for them and they are never written out), else 16-byte copies zero-filled
        // past its tokens, handed to the async proxy
        uint32_t qn = 0;
        bool ok = p.q != nullptr;
        for (int rnd = 0, item; ok && (item = snake_item(rnd, n_items)) >= 0; ++rnd) {
            const Work w = item_work(rnd, item);
            if (w.nkeys <= 0) continue;
            if (lane == 0) ok = mbar_wait(q_empty, (qn & 1u) ^ 1u, p.status, abort_flag);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            const int64_t tok0 = w.tok0;
            const uint32_t dst0 = smem_addr(sQ);
            if (tok0 + p.tq <= p.total_q) {
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
                const bool valid = t_row < w.ntok;
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
        // members whose rows differ from their group's first over the shared blocks
        for (int s = blockIdx.x; p.own && s < p.num_seqs; s += gridDim.x) {
            const Group g = group_of_seq(p, s);
            if (!g.shares || s == g.b0) continue;
            const int32_t* first = p.block_table + static_cast<int64_t>(g.b0) * p.max_blocks;
            const int32_t* mine = p.block_table + static_cast<int64_t>(s) * p.max_blocks;
            bool differs = false;
#pragma unroll 4
            for (int j = lane; j < g.s0 / p.block_size; j += 32) differs |= __ldg(first + j) != __ldg(mine + j);
            if (differs) report(p.status, PA_ERR_INVALID_ARG);
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
        const uint64_t dk = smem_desc(smem_addr(sK), 16, kGroupBytes);
        const uint64_t dv = smem_desc(smem_addr(sV), kGroupBytes / 2, kGroupBytes);
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
                    // Q and K: 32 bytes per k-step in a 64-column half
                    mma_f16_ss(tmem + kColS + b * kBN, dq + (k / 4) * (kBlkBytes >> 4) + (k % 4) * 2,
                               dks + (k / 4) * (kGroupBytes >> 5) + (k % 4) * 2, id_qk, k > 0 ? 1u : 0u);
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
                const int ntiles = w_next.tiles();
                const int item2 = snake_item(rnd + 1, n_items);
                if (ntiles == 0) {
                    item = item2;
                    if (item >= 0) w_next = item_work(rnd + 1, item);
                    continue;
                }
                ok = mbar_wait(q_full, q_cnt & 1u, p.status, abort_flag);
                const uint32_t col_o = tmem + kColO + (q_cnt & 1u) * kD;  // this item's O
                ++q_cnt;
                if (ok) ok = issue_qk(0, ntiles == 1);
                if (ok && ntiles > 1) ok = issue_qk(1, ntiles == 2);
                item = item2;
                if (item >= 0) w_next = item_work(rnd + 1, item);
                for (int t = 0; t < ntiles && ok; ++t) {
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
                            // V: two groups per 16 keys
                            mma_f16_ts(col_o, tmem + kColS + y * kBN + (j / 4) * 64 + part * 32 + (j % 4) * 8,
                                       dvs + j * (2 * kGroupBytes >> 4), id_pv, (t > 0 || part > 0 || j > 0) ? 1u : 0u);
                        }
                    }
                    mma_commit(v_empty + 8 * v_stage);
                    mma_commit(o_done + 8 * (pv_count & 1u));
                    ++pv_count;
                    if (++v_stage == kStagesV) {
                        v_stage = 0;
                        v_phase ^= 1u;
                    }
                    if (t + 2 < ntiles) ok = issue_qk(t + 2, t + 3 == ntiles);
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
        // where this row of item w goes: its offset in out (>= 0), or -2 - its slot in
        // the workspace, or -1 for no row
        auto row_of = [&](const Work& w) -> int64_t {
            const int t_row = r / p.group, g_row = r - t_row * p.group;
            if (t_row >= w.ntok) return -1;
            const int64_t row = static_cast<int64_t>(w.tok0 + t_row) * p.num_heads + w.kvh * p.group + g_row;
            return w.part < 0 ? row * kD : -2 - (row * p.max_parts + w.part);
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
                // (a warp's rows go one way: tensor memory is read by whole warps)
                if (__any_sync(0xffffffffu, my_off <= -2)) {
                    // a part: O / l in 32 bits, and log2 of the sum of 2^score
                    const int64_t slot = -2 - my_off;
                    if (x == 0 && my_off <= -2) p.ws_lse[slot] = L > 0.f ? pend_m[u] + __log2f(L) : -INFINITY;
                    float* dst_f = p.ws_o + slot * kD + 64 * x;
#pragma unroll
                    for (int c0 = 0; c0 < 64; c0 += 32) {
                        float o[32];
                        tmem_ld32(o_col + c0, o);
                        uint32_t wv[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) wv[j] = __float_as_uint(o[j] * inv);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (my_off <= -2) st_global_v8(dst_f + c0 + 8 * j, wv + 8 * j);
                    }
                } else if (__any_sync(0xffffffffu, my_off >= 0)) {
                    uint16_t* dst_e = static_cast<uint16_t*>(p.out) + my_off + 64 * x;
                    // 32-byte stores (whole sectors) when out allows them
                    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
#pragma unroll
                    for (int c0 = 0; c0 < 64; c0 += 32) {
                        float o[32];
                        tmem_ld32(o_col + c0, o);
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
            const int ntiles = w.tiles();
            const int64_t row_off = row_of(w);
            const int t_row = r / p.group;
            // visible keys of this row: [0, lim)
            const int lim = t_row < w.ntok ? min(w.nkeys, w.shift + t_row + 1) : 0;
            if (ntiles == 0 && !end) {
                // no visible key for any row of the item: output 0 (a part: the merge
                // does not read it)
                if (row_off >= 0) {
                    uint16_t* dst = static_cast<uint16_t*>(p.out) + row_off + 64 * x;
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
                if (t >= ntiles) break;
                const int b = t & 1;
                const int key0 = t * kBN + 64 * x;  // first key of this thread's 64 columns
                const int vis = lim - key0;  // visible keys of these columns: [0, vis)
                ok = ok && mbar_wait(s_full + 8 * b, s_use[b] & 1u, p.status, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();  // for both reads of S below
                ++s_use[b];
                float e[64];
                float sum = 0.f;
                bool over = false;
                // (an item's first tile has no reference: straight to the true maximum)
                const bool first = t == 0;
                if (ok && !first) {
                    tmem_ld64(sbuf + b * kBN, e);
                    hide_keys(e, vis);
                    if (m == -INFINITY) {
                        // no reference yet: the slow path, unless these columns
                        // are all masked for this row (weights 0)
                        over = vis > 0;
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
                        hide_keys(e, vis);
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
                // values past the last key may hold anything: zero those V rows (after
                // the tile landed) so zero weights never meet NaN
                if (t * kBN + kBN > w.nkeys) {
                    const uint32_t f = tiles + t;
                    ok = mbar_wait(v_full + 8 * (f % kStagesV), (f / kStagesV) & 1u, p.status, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) continue;
                    uint8_t* vt = sV + (f % kStagesV) * kTileBytes;
                    const int rest = w.nkeys - t * kBN;
                    for (int ci = u; ci < (kBN - rest) * 16; ci += 256) {
                        const int rr = rest + (ci >> 4), c = ci & 15;
                        *reinterpret_cast<uint4*>(vt + (rr >> 3) * kGroupBytes + (c >> 3) * (kGroupBytes / 2) + sw128(rr & 7, c & 7)) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
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
            tiles += ntiles;
            pend = true;
            pend_ok = ok;
            pend_l[u] = l;
            pend_m[u] = m;
            pend_off[u] = row_off;
        }
    }
    // ---- teardown: every role is done; free tensor memory ----
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

// The rows that have parts: a warp takes a (query row, head), a lane four columns.
template <int DT>
__global__ void __launch_bounds__(256) cascade_merge_kernel(const CascadeParams p) {
    pdl_trigger();
    // (The lengths are the call's inputs: the kernels before this one had waited for what
    // wrote them before they let it start.  Every warp waits, also one that has nothing to
    // do: what comes after this kernel counts on the ones before it being done.)
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    int q0, lq, lk;
    if (!seq_lens_ok(p, b, q0, lq, lk)) return pdl_wait();
    const int64_t pair = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (pair >= static_cast<int64_t>(lq) * p.num_heads) return pdl_wait();
    const Group g = group_of_seq(p, b);
    if (!g.ok || g.s0 > lk - lq) return pdl_wait();
    const int start = g.shares ? g.s0 : 0;
    if (p.own && start == 0 && lk <= p.part) return pdl_wait();  // one part, already in out
    const int i = static_cast<int>(pair / p.num_heads);
    const int seen = lk - lq + i + 1 - start;  // own keys
    // (its tile among the group's)
    const bool tail = start > 0 && (q0 - __ldg(p.cu_q + g.b0) + i) / p.tq >= p.tail_from;
    const int pre = start > 0 ? ceil_div(start, tail ? p.tail_part : p.part) : 0;
    const int np = pre + (seen > 0 ? ceil_div(seen, p.own ? p.part : p.own_part) : 0);
    const int skip = start > 0 || !p.own ? p.own_base - pre : 0;  // numbers between the prefix's parts and the own keys'
    const int64_t row = static_cast<int64_t>(q0) * p.num_heads + pair;
    const float* lse = p.ws_lse + row * p.max_parts;
    const float4* o = reinterpret_cast<const float4*>(p.ws_o + row * p.max_parts * kD) + lane;
    pdl_wait();
    float M = -INFINITY;
    for (int j = lane; j < np; j += 32) M = fmaxf(M, lse[j < pre ? j : j + skip]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    if (M > -INFINITY) {
#pragma unroll 4
        for (int j = 0; j < np; ++j) {
            const int at = j < pre ? j : j + skip;
            const float w = ex2(lse[at] - M);
            const float4 v = o[static_cast<int64_t>(at) * (kD / 4)];
            sum += w;
            acc.x = fmaf(w, v.x, acc.x);
            acc.y = fmaf(w, v.y, acc.y);
            acc.z = fmaf(w, v.z, acc.z);
            acc.w = fmaf(w, v.w, acc.w);
        }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * kD + 4 * lane) =
        make_uint2(pack2<DT>(acc.x * inv, acc.y * inv), pack2<DT>(acc.z * inv, acc.w * inv));
}

// The SMs of a GB300, whatever the device: the workspace query needs none.
constexpr int kSms = 152;

struct Plan {
    bool stack, own;
    int part, tail_from, tail_part, max_parts, own_base;
    size_t o_off, lens_off, bytes;
};
constexpr int kOwnPart = 1024;  // the decode kernel's parts

// How the batch is cut, from what the host knows of it.
//
// Stacking.  Sequences whose queries fill two tiles or more each gain little from standing
// together, and their rows' parts cost a write, a read and a merge: they take their keys as
// one segment straight to out.  (Four system prompts of 1024 to 8192 tokens, 20 prompts of
// 16 to 1024 tokens behind them, 32/8 heads, bf16: 1069 us stacked, 832
// not.)  With few query tiles over long keys they are cut into parts all the same.
//
// Own keys of one-token sequences.  A tile of 128 rows for one query token's heads pays its
// start and end (some 5 us, few of them hidden) for a handful of keys: past one round of
// items they go to the decode kernel, which takes the same slots.  (32 requests of eight beams,
// up to 256 tokens of their own: 159 us in tiles, 142 by the decode kernel.)
//
// Parts.  n parts of the longest prefix make tiles * n items for the SMs' rounds; an item
// costs its key tiles and some 2.5 more for its start and end, a part's rows 1 KB of traffic
// a row and head.  The n with the least such time is taken.
Plan plan_of(int64_t num_seqs, int64_t num_groups, int64_t total_q, int num_heads, int num_kv_heads, int max_q, int max_k, int max_shared) {
    Plan r;
    const int group = num_heads / num_kv_heads;
    r.stack = max_shared > 0 && total_q * group < 2ll * kRows * num_seqs;
    int64_t row_tiles = (total_q * group + kRows - 1) / kRows;
    if (r.stack && row_tiles < num_groups) row_tiles = num_groups;  // (no tile is of two groups)
    const int64_t tiles = row_tiles * num_kv_heads;
    const int keys = r.stack ? max_shared : max_k;
    const double rows_us = static_cast<double>(total_q) * num_heads * 1032.0 / 6.5e6;  // a part's traffic
    const int key_tiles = (keys + kBN - 1) / kBN > 0 ? (keys + kBN - 1) / kBN : 1;
    auto size_of = [&](int n) { return (key_tiles + n - 1) / n > 2 ? (key_tiles + n - 1) / n : 2; };  // key tiles of n parts
    auto rounds = [&](double items) { return std::ceil(items / kSms); };
    double best = -1.0;
    r.tail_from = INT32_MAX;
    r.part = r.tail_part = kBN;
    for (int n = 1; n <= 64; ++n) {
        const int size = size_of(n);
        const double merge = n > 1 || r.stack ? (n + 1) * rows_us : 0.0;
        double t = rounds(static_cast<double>(tiles) * n) * 1.3 * (size + 2.5) + merge;
        if (num_groups > 1) {
            // prefixes of unlike length, half of the longest on average: the longest items
            // first, half an item's time uneven at the end
            const double mean = tiles * (0.5 * key_tiles + 2.5 * (0.5 * n + 0.5)) / kSms + 0.5 * (size + 2.5);
            t = 1.3 * (mean > size + 2.5 ? mean : size + 2.5) + 0.5 * merge;
        }
        if (best < 0.0 || t < best) {
            best = t;
            r.part = r.tail_part = size * kBN;
            r.tail_from = INT32_MAX;
        }
        // one group: whole rounds of such parts, and the query tiles of the last,
        // partly filled round in parts of their own
        const int64_t rows = row_tiles, whole = tiles * n / kSms;
        const int64_t from = whole * kSms / (static_cast<int64_t>(num_kv_heads) * n);
        if (r.stack && num_groups == 1 && n <= 8 && from > 0 && from < rows)
            for (int m = n + 1; m <= 24; ++m) {
                const int small = size_of(m);
                const double u = rounds(static_cast<double>(from) * num_kv_heads * n) * 1.3 * (size + 2.5) +
                                 rounds(static_cast<double>(rows - from) * num_kv_heads * m) * 1.3 * (small + 2.5) + merge +
                                 (m - n) * rows_us * (rows - from) / rows;
                if (u < 0.97 * best) {
                    best = u;
                    r.part = size * kBN;
                    r.tail_from = static_cast<int>(from);
                    r.tail_part = small * kBN;
                }
            }
        if (size == 2) break;
    }
    r.own = !(r.stack && max_q == 1 && total_q >= num_seqs && (tiles + num_seqs * num_kv_heads) > kSms);
    const int least = r.tail_part < r.part ? r.tail_part : r.part;
    r.own_base = (max_shared + least - 1) / least;
    // (not stacked and one part: everything goes straight to out)
    r.max_parts = !r.own                          ? r.own_base + (max_k + kOwnPart - 1) / kOwnPart
                  : !r.stack && max_k <= r.part ? 1
                                                  : (r.stack ? r.own_base : 0) + (max_k + r.part - 1) / r.part;
    r.o_off = r.lens_off = r.bytes = 0;
    if (r.max_parts == 1) return r;
    const size_t rows = static_cast<size_t>(total_q) * num_heads * r.max_parts;
    r.o_off = (rows * 4 + 255) & ~static_cast<size_t>(255);
    r.lens_off = r.o_off + rows * kD * 4;
    r.bytes = r.lens_off + (r.own ? 0 : static_cast<size_t>(num_seqs) * 4) + 16;  // (32-byte stores: the pointer is rounded up)
    return r;
}

template <int DT>
pa_status launch_cascade(CascadeParams p, const void* q, const pa_kv_cache& cache, const CUtensorMap& map_k, const CUtensorMap& map_v, const CUtensorMap& map_q,
                         cudaStream_t stream) {
    const int n_seg = p.num_groups + (p.own ? p.num_seqs : 0);
    const int base = kSmemBytes + (n_seg + 1) * 4 + 1024;
    if (base > device_max_smem_optin()) return PA_ERR_UNSUPPORTED;
    // an upper bound of the entries: every query tile with every part
    const int64_t tiles = static_cast<int64_t>(p.total_q) / p.tq + p.num_groups + (p.own ? p.num_seqs : 0);
    const int64_t bound = tiles * p.max_parts;
    // (2 KB kept back for the kernel's static shared memory)
    const int64_t room = (device_max_smem_optin() - 2048 - base) / 4 - (kThreads / 32) * 64;
    p.order_cap = static_cast<int32_t>(room <= 0 ? 0 : (bound < room ? bound : room));
    const int smem = base + (p.order_cap > 0 ? (p.order_cap + (kThreads / 32) * 64) * 4 : 0);
    static LaunchCache launch_cache;
    auto kern = cascade_kernel<DT>;
    const int per_sm = blocks_per_sm(kern, kThreads, smem, launch_cache);
    if (per_sm <= 0) return PA_ERR_CUDA;
    const int64_t max_items = bound * p.num_kv_heads;
    const int64_t cap = static_cast<int64_t>(device_sm_count()) * per_sm;
    const int grid = static_cast<int>(max_items < cap ? max_items : cap);
    if (grid > 0 && launch_pdl(kern, grid, kThreads, smem, stream, map_k, map_v, map_q, p) != cudaSuccess) return PA_ERR_CUDA;
    if (p.max_parts == 1) return PA_OK;
    if (!p.own) {
        DecodeParams d{};
        d.q = q;
        d.k_cache = static_cast<const uint8_t*>(cache.k_cache);
        d.v_cache = static_cast<const uint8_t*>(cache.v_cache);
        d.block_table = p.block_table;
        d.seq_lens = p.ws_lens;
        d.ws_lse = p.ws_lse;
        d.ws_o = p.ws_o;
        d.status = p.status;
        d.num_blocks = p.num_blocks;
        d.block_size = p.block_size;
        d.num_kv_heads = p.num_kv_heads;
        d.num_heads = p.num_heads;
        d.num_seqs = d.num_members = p.num_seqs;
        d.max_blocks = p.max_blocks;
        d.max_seq_len = p.max_k;
        d.partition = p.own_part;
        d.max_parts = p.max_parts;
        d.qk_scale = p.scale_log2;
        d.v_scale = d.k_scale_w = d.v_scale_w = 1.f;
        d.cu_groups = p.cu_groups;
        d.shared_lens = p.shared_lens;
        d.num_groups = p.num_groups;
        d.own_base = p.own_base;
        pa_status (*const launch[2][3])(const DecodeParams&, int, int, int, cudaStream_t) = {
            {launch_decode_f16_bs16, launch_decode_f16_bs32, launch_decode_f16_bs64},
            {launch_decode_bf16_bs16, launch_decode_bf16_bs32, launch_decode_bf16_bs64}};
        const pa_status st = launch[DT == PA_BF16][p.block_size == 16 ? 0 : p.block_size == 32 ? 1 : 2](d, DT, kD, p.group, stream);
        if (st != PA_OK) return st;
    }
    const int64_t per_seq = (static_cast<int64_t>(p.max_q) * p.num_heads + 7) / 8;
    if (per_seq > INT32_MAX) return PA_ERR_UNSUPPORTED;
    const dim3 mgrid(static_cast<unsigned>(per_seq), static_cast<unsigned>(p.num_seqs));
    return launch_pdl(cascade_merge_kernel<DT>, mgrid, 256, 0, stream, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_varlen_cascade_workspace_size(int32_t num_seqs, int64_t total_q, int32_t num_heads,
                                                   int32_t num_kv_heads, int32_t head_size, int32_t max_seqlen_q,
                                                   int32_t max_seqlen_k, int32_t max_shared_len, int32_t block_size) {
    if (num_seqs <= 0 || total_q <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 ||
        head_size <= 0 || max_seqlen_q <= 0 || max_seqlen_k < 0 || max_shared_len < 0 || block_size <= 0)
        return 0;
    // (the groups are not told here: the larger of the two ways)
    const size_t a = plan_of(num_seqs, 1, total_q, num_heads, num_kv_heads, max_seqlen_q, max_seqlen_k, max_shared_len).bytes;
    const size_t b = plan_of(num_seqs, 2, total_q, num_heads, num_kv_heads, max_seqlen_q, max_seqlen_k, max_shared_len).bytes;
    return a > b ? a : b;
}

namespace {

// pa_varlen_cascade; no_copies: the test hook's launch
pa_status cascade_entry(void* out, const void* q, pa_dtype q_dtype, const pa_kv_cache* cache,
                        const int32_t* block_table, int32_t max_blocks_per_seq,
                        const int32_t* cu_seq_lens_q, const int32_t* cu_seq_lens_k, int32_t num_seqs,
                        int64_t total_q, int32_t max_seqlen_q, int32_t max_seqlen_k, int32_t num_heads,
                        float scale, const int32_t* cu_groups, const int32_t* shared_lens,
                        int32_t num_groups, int32_t max_group_size, int32_t max_shared_len,
                        void* workspace, size_t workspace_bytes, int32_t* dev_status,
                        pa_stream_t stream, bool no_copies) {
    const pa_status st = check_cache(cache);
    if (st != PA_OK) return st;
    if (num_seqs < 0 || num_groups < 0 || num_heads <= 0 || max_blocks_per_seq <= 0 || total_q < 0 || max_seqlen_q < 0 ||
        max_seqlen_k < 0 || max_group_size < 0 || max_shared_len < 0 || max_shared_len > max_seqlen_k ||
        max_shared_len % cache->block_size != 0)
        return PA_ERR_INVALID_ARG;
    // (the running maximum is taken over unscaled scores)
    if (!(scale > 0.f) || !std::isfinite(scale)) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || max_seqlen_q == 0 || total_q == 0) return PA_OK;
    if (out == nullptr || q == nullptr || block_table == nullptr || cu_seq_lens_q == nullptr ||
        cu_seq_lens_k == nullptr || cu_groups == nullptr || shared_lens == nullptr || num_groups == 0)
        return PA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(out) & 15u) || (reinterpret_cast<uintptr_t>(q) & 15u)) return PA_ERR_INVALID_ARG;
    if (num_heads % cache->num_kv_heads != 0) return PA_ERR_INVALID_ARG;
    const int group = num_heads / cache->num_kv_heads;
    if (cache->head_size != kD) return PA_ERR_UNSUPPORTED;
    if (group != 1 && group != 2 && group != 4 && group != 8) return PA_ERR_UNSUPPORTED;
    if (q_dtype != PA_F16 && q_dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (cache->kv_dtype != q_dtype) return PA_ERR_UNSUPPORTED;
    const int bs = cache->block_size;
    if (bs != 16 && bs != 32 && bs != 64) return PA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(num_seqs) + num_groups > kMaxSegments) return PA_ERR_UNSUPPORTED;
    const int64_t rows = cache->num_blocks * cache->num_kv_heads * bs;
    if (rows > INT32_MAX || total_q > INT32_MAX - kRows) return PA_ERR_UNSUPPORTED;
    Plan plan = plan_of(num_seqs, num_groups, total_q, num_heads, cache->num_kv_heads, max_seqlen_q, max_seqlen_k, max_shared_len);
    // (never more than the workspace query's answer)
    if (plan.bytes > pa_varlen_cascade_workspace_size(num_seqs, total_q, num_heads, cache->num_kv_heads, kD, max_seqlen_q,
                                                      max_seqlen_k, max_shared_len, bs))
        plan = plan_of(num_seqs, 2, total_q, num_heads, cache->num_kv_heads, max_seqlen_q, max_seqlen_k, max_shared_len);
    if (plan.bytes > 0 && (workspace == nullptr || workspace_bytes < plan.bytes || (reinterpret_cast<uintptr_t>(workspace) & 15u)))
        return PA_ERR_INVALID_ARG;

    CascadeParams p{};
    p.out = out;
    p.q = no_copies ? nullptr : static_cast<const uint16_t*>(q);
    p.block_table = block_table;
    p.cu_q = cu_seq_lens_q;
    p.cu_k = cu_seq_lens_k;
    p.cu_groups = cu_groups;
    p.shared_lens = shared_lens;
    char* ws = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(workspace) + 31u) & ~uintptr_t{31u});
    p.ws_lse = reinterpret_cast<float*>(ws);
    p.ws_o = reinterpret_cast<float*>(ws + plan.o_off);
    p.status = dev_status;
    p.num_blocks = cache->num_blocks;
    p.block_size = bs;
    p.num_kv_heads = cache->num_kv_heads;
    p.num_heads = num_heads;
    p.group = group;
    p.tq = kRows / group;
    p.num_seqs = num_seqs;
    p.num_groups = num_groups;
    p.max_blocks = max_blocks_per_seq;
    p.max_q = max_seqlen_q;
    p.max_k = max_seqlen_k;
    p.max_group = max_group_size;
    p.max_shared = max_shared_len;
    p.total_q = static_cast<int32_t>(total_q);
    p.part = plan.part;
    p.tail_from = plan.tail_from;
    p.tail_part = plan.tail_part;
    p.max_parts = plan.max_parts;
    p.own = plan.own ? 1 : 0;
    p.own_base = plan.own_base;
    p.own_part = kOwnPart;
    p.ws_lens = reinterpret_cast<int32_t*>(ws + plan.lens_off);
    p.stack = plan.stack ? 1 : 0;
    p.scale_log2 = scale * 1.4426950408889634f;
    CUtensorMap map_k, map_v, map_q;
    if (!make_page_map(&map_k, cache->k_cache, rows, q_dtype, bs) ||
        !make_page_map(&map_v, cache->v_cache, rows, q_dtype, bs) ||
        !make_q_map(&map_q, q, num_heads, group, p.total_q, q_dtype))
        return PA_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return q_dtype == PA_BF16 ? launch_cascade<PA_BF16>(p, q, *cache, map_k, map_v, map_q, s)
                              : launch_cascade<PA_F16>(p, q, *cache, map_k, map_v, map_q, s);
}

}  // namespace

extern "C" pa_status pa_varlen_cascade(void* out, const void* q, pa_dtype q_dtype, const pa_kv_cache* cache,
                                       const int32_t* block_table, int32_t max_blocks_per_seq,
                                       const int32_t* cu_seq_lens_q, const int32_t* cu_seq_lens_k, int32_t num_seqs,
                                       int64_t total_q, int32_t max_seqlen_q, int32_t max_seqlen_k, int32_t num_heads,
                                       float scale, const int32_t* cu_groups, const int32_t* shared_lens,
                                       int32_t num_groups, int32_t max_group_size, int32_t max_shared_len,
                                       void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                       pa_stream_t stream) {
    return cascade_entry(out, q, q_dtype, cache, block_table, max_blocks_per_seq, cu_seq_lens_q, cu_seq_lens_k, num_seqs, total_q,
                         max_seqlen_q, max_seqlen_k, num_heads, scale, cu_groups, shared_lens, num_groups, max_group_size,
                         max_shared_len, workspace, workspace_bytes, dev_status, stream, false);
}

extern "C" pa_status pa_varlen_cascade_test_wait_timeout(void* out, const void* q, pa_dtype q_dtype, const pa_kv_cache* cache,
                                       const int32_t* block_table, int32_t max_blocks_per_seq,
                                       const int32_t* cu_seq_lens_q, const int32_t* cu_seq_lens_k, int32_t num_seqs,
                                       int64_t total_q, int32_t max_seqlen_q, int32_t max_seqlen_k, int32_t num_heads,
                                       float scale, const int32_t* cu_groups, const int32_t* shared_lens,
                                       int32_t num_groups, int32_t max_group_size, int32_t max_shared_len,
                                       void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                       pa_stream_t stream) {
    return cascade_entry(out, q, q_dtype, cache, block_table, max_blocks_per_seq, cu_seq_lens_q, cu_seq_lens_k, num_seqs, total_q,
                         max_seqlen_q, max_seqlen_k, num_heads, scale, cu_groups, shared_lens, num_groups, max_group_size,
                         max_shared_len, workspace, workspace_bytes, dev_status, stream, true);
}
