// Norms of the queries and keys of each head, the position rotation and the
// cache write, in one pass over the projections' output.
//
// For a head's row x of D elements (D = head size), with weight w and eps:
//     y = x / sqrt(mean(x^2) + eps) * w               (no weight: y = x)
// and for pair i of its first `rotary_dim` elements (a = i, b = i +
// rotary_dim/2 in the half layout; a = 2i, b = 2i+1 interleaved), at position
// p and theta_i radians per position, f the rope factor:
//     out_a = f (y_a cos(p theta_i) - y_b sin(p theta_i))
//     out_b = f (y_b cos(p theta_i) + y_a sin(p theta_i)),
// the other elements as they are.  Sums and products are in fp32; the result is
// rounded once, to the output's type (an E4M3 cache: satfinite(rne(out / scale))
// of the fp32 value, not of a 16-bit one in between).  Value rows go to the cache
// as pa_kv_cache_write stores them.
//
// Angles: frequencies are turns per position in units of 2^-64, so position *
// frequency wraps to the exact fraction of a turn, whose top 32 bits go to
// sincospif: no table to read, and no position too far.
//
// The kernel is bandwidth-bound (2 bytes in and 2 or 1 out per element) as long
// as it spends few instructions on an element: a first version with 8 elements
// a lane took 172 instructions for 256 elements and was bound by their issue
// at 70 % of the copy rate.  So D/16 lanes share a row, two 16-byte chunks a
// lane, chosen so that a lane holds both elements of its pairs: chunks j and j +
// rotary_dim/16 in the half layout (the lanes past the rotated part share the
// rest), whole pairs in any chunk when interleaved.  No element changes lanes,
// the sum of squares is all that does.  A warp takes a step of 4 heads (8 of
// 64 elements) at a time.  The resident warps take a token each, round by
// round, and the last round's steps (what its tokens have of queries, keys and
// values) are dealt out in equal runs.  Each lane keeps
// the next rows in flight through a ring of its own in shared memory (16-byte
// asynchronous copies that only the same lane reads back: no barrier, and no
// register held while a load is on its way).  When a run enters a token, the warp
// works out its sines (two per lane, exchanged through shared memory) and folds
// the norm's weights into them:
//     out = r (x w cos + x' w' sin),  r = 1 / sqrt(mean(x^2) + eps),
// with x' the other element of the pair.
//
// On one GB300: 16384 tokens of 32/8 heads of 128 (bf16, normed, into the cache) in
// 64.7 us, 6.2 TB/s, 0.92 of the measured copy rate (238 instructions a step of 512
// elements, 64 % of the issue slots); 5461 tokens of 32/32 heads (fp16, rotation alone,
// packed) in 30.5 us, 5.9 TB/s; one token in 2.7 us, a launch and one dependent chain.
#include <cmath>

#include "common.cuh"
#include "launch.h"

namespace pa {
namespace {

constexpr int kWarps = 4;    // warps of a block
constexpr int kBlocks = 4;   // blocks per SM that the registers allow
constexpr int kDepth = 4;    // steps a lane's ring holds
constexpr int kPacked = -1;  // keys go to packed rows, there is no cache

struct NormRopeParams {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* q_out;
    void* k_out;  // packed rows, or the K cache
    void* v_out;  // the V cache
    int64_t q_stride, k_stride, v_stride, qo_stride, ko_stride;  // elements from token to token
    const int64_t* positions;
    const int64_t* slots;
    const uint64_t* turns;
    const float* q_weight;
    const float* k_weight;
    int32_t* status;
    int64_t num_tokens;
    int64_t num_slots;
    float eps, rope_factor, k_scale, v_scale;
    float k_inverse, v_inverse;  // 1 / scale where the scale is a power of two, else 0
    int32_t num_heads, num_kv_heads;
    int32_t rotary_dim, interleaved, block_size;
    // each warp takes tokens w, w + warps, ... for `rounds` rounds, then a run of
    // the remaining tokens' steps: per_warp, one more for the first `extra` warps
    int64_t warps, rounds, per_warp, extra;
    // 16-byte accesses allowed (pointer and stride aligned)
    bool q_vec, k_vec, v_vec, qo_vec, ko_vec;
};

// 16 bytes of a row that is not 16-byte aligned
__device__ __forceinline__ uint4 load_odd8(const uint16_t* p) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = static_cast<uint32_t>(p[2 * j]) | static_cast<uint32_t>(p[2 * j + 1]) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store_row8(uint16_t* p, uint4 x, bool vec) {
    if (vec) {
        *reinterpret_cast<uint4*>(p) = x;
        return;
    }
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        p[2 * j] = static_cast<uint16_t>(w[j]);
        p[2 * j + 1] = static_cast<uint16_t>(w[j] >> 16);
    }
}

template <int DT>
__device__ __forceinline__ uint32_t round_pair(float a, float b) {
    if constexpr (DT == PA_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

// packed fp32 pairs: one instruction for both halves
__device__ __forceinline__ uint64_t pair2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpair2(uint64_t r) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(r));
    return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
template <int DT>
__device__ __forceinline__ uint64_t widen(uint32_t w) {
    const float2 f = kv_pair<DT>(w);
    return pair2(f.x, f.y);
}

// 8 values (packed pairs) -> 8 E4M3 codes: IEEE division, then one rounding with
// saturation.  (By a power of two, x / scale and x * (1 / scale) are the same
// number rounded once.  16 divisions a lane by other scales: 256 tokens, 32/8 heads,
// 5.0 us for 3.9; 16384 tokens, normed, 83 us for 67.)
__device__ __forceinline__ uint2 e4m3_8(const uint64_t* x, float scale, float inverse) {
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float2 f = unpair2(x[j]);
        if (inverse != 0.f) f = unpair2(mul2(x[j], pair2(inverse, inverse)));
        else f = make_float2(__fdiv_rn(f.x, scale), __fdiv_rn(f.y, scale));
        c[j] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3));
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
template <int DT>
__device__ __forceinline__ uint4 round_8(const uint64_t* x) {
    uint32_t y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = unpair2(x[j]);
        y[j] = round_pair<DT>(f.x, f.y);
    }
    return make_uint4(y[0], y[1], y[2], y[3]);
}

// A warp's tokens in turn: one a round, then those of its last run.
struct Tokens {
    int64_t t, round, last;  // last: the last run's first token
    __device__ __forceinline__ int64_t after(const NormRopeParams& p) const {
        return round + 1 < p.rounds ? t + p.warps : round + 1 == p.rounds ? last : t + 1;
    }
    __device__ __forceinline__ void next(const NormRopeParams& p) {
        t = after(p);
        ++round;
    }
};

// The rows that a warp loads: a cursor over (token, segment, step), the
// segments of a token being its queries (0), keys (1) and values (2).
template <int KVT, int D>
struct Loader {
    static constexpr int RPS = 512 / D;  // rows of a step
    static constexpr int kSegs = KVT == kPacked ? 2 : 3;
    const uint16_t* src;  // this lane's first chunk of the step's row
    Tokens at;
    int64_t left;  // steps not yet issued
    int first_seg, first_step;  // where the last run begins in its token
    int rows;      // rows of the segment from this lane's on
    int seg;
    bool vec;

    __device__ __forceinline__ void enter(const NormRopeParams& p, int step, int sub, int c0) {
        const uint16_t* base = seg == 0   ? p.q + at.t * p.q_stride
                               : seg == 1 ? p.k + at.t * p.k_stride
                                          : p.v + at.t * p.v_stride;
        vec = seg == 0 ? p.q_vec : seg == 1 ? p.k_vec : p.v_vec;
        rows = (seg == 0 ? p.num_heads : p.num_kv_heads) - step * RPS - sub;
        src = base + (step * RPS + sub) * D + c0 * 8;
    }
    // starts the copies of the next step's row into `slot` and slot[32] (one
    // group of asynchronous copies a step, empty past the run's end); the second
    // chunk is `gap` elements after the first
    __device__ __forceinline__ void issue(const NormRopeParams& p, uint4* slot, int sub, int c0, int gap) {
        if (left > 0) {
            const bool have = rows > 0;
            if (vec) {
                // (nothing is read for a row past the segment's, but its address has
                // to be an aligned one, which q's need not be here)
                const uint64_t nowhere = reinterpret_cast<uint64_t>(p.q) & ~uint64_t{15};
                const uint64_t from = have ? reinterpret_cast<uint64_t>(src) : nowhere;
                const uint64_t from1 = have ? reinterpret_cast<uint64_t>(src + gap) : nowhere;
                const uint32_t n = have ? 16u : 0u;
                asm volatile(
                    "cp.async.cg.shared.global [%0], [%1], 16, %3;\n\t"
                    "cp.async.cg.shared.global [%0 + 512], [%2], 16, %3;" ::"r"(smem_addr(slot)),
                    "l"(from), "l"(from1), "r"(n)
                    : "memory");
            } else {
                slot[0] = have ? load_odd8(src) : make_uint4(0u, 0u, 0u, 0u);
                slot[32] = have ? load_odd8(src + gap) : make_uint4(0u, 0u, 0u, 0u);
            }
            --left;
            src += RPS * D;
            rows -= RPS;
            // (the segment's last step: no row is left for the step's first lanes)
            if (rows + sub <= 0 && left > 0) {
                int step = 0;
                if (++seg == kSegs) {
                    seg = 0;
                    at.next(p);
                    if (at.round == p.rounds) {
                        seg = first_seg;
                        step = first_step;
                    }
                }
                enter(p, step, sub, c0);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
};

// What a warp's run works on: its token, this lane's place in the rows, the
// ring, the token's sines once they are worked out.
template <int KVT, int D>
struct Run {
    Loader<KVT, D> load;
    uint4* ring;      // [kDepth][2][32], this lane's slots
    int slot;         // of the step to work on
    Tokens tok;
    int64_t at;       // cache row of the token's KV head 0, -1 for none
    float2* turn;     // shared memory: (cos, sin) * factor of the token's pairs
    int64_t pos, next_pos;
    int64_t next_slot;
    int sub;          // row of a step
    int c0, gap;      // first chunk of 8 elements; elements from it to the second
    int half;         // chunks of half the rotated part
    bool turned0, turned1;  // the chunks lie in the rotated part
    bool ready;       // the sines are in `turn`
};

// (cos, sin) of the token's pairs into shared memory, once a token
template <int KVT, int D>
__device__ __forceinline__ void work_out_sines(const NormRopeParams& p, Run<KVT, D>& u) {
    if (u.ready || u.half == 0) return;
    u.ready = true;
    __syncwarp();  // (the token before may still be read)
    for (int i = threadIdx.x & 31; i < p.rotary_dim / 2; i += 32) {
        // the signed top half of the phase is the fraction of a turn in units
        // of 2^-32, so * 2^-31 gives half turns in [-1, 1)
        const int32_t frac = static_cast<int32_t>((static_cast<uint64_t>(u.pos) * __ldg(p.turns + i)) >> 32);
        float s, c;
        sincospif(static_cast<float>(frac) * 4.656612873077393e-10f, &s, &c);
        u.turn[i] = make_float2(c * p.rope_factor, s * p.rope_factor);
    }
    __syncwarp();
}

// The token's position and its slot's place in the cache (loaded a token ahead).
template <int KVT, int D>
__device__ __forceinline__ void enter_token(const NormRopeParams& p, Run<KVT, D>& u) {
    u.ready = false;
    u.pos = u.next_pos;
    const int64_t slot = u.next_slot;
    const int64_t after = u.tok.after(p);
    if (after < p.num_tokens) {
        if (u.half > 0) u.next_pos = __ldg(p.positions + after);
        if (KVT != kPacked) u.next_slot = __ldg(p.slots + after);
    }
    if (KVT != kPacked) {
        u.at = -1;
        if (slot >= p.num_slots) {
            if ((threadIdx.x & 31) == 0) report(p.status, PA_ERR_BAD_BLOCK);
        } else if (slot >= 0) {
            // (a 32-bit division where it does: a 64-bit one is ten times as long)
            const int64_t blk = slot >> 32 == 0 ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.block_size)
                                                : slot / p.block_size;
            u.at = blk * p.num_kv_heads * p.block_size + (slot - blk * p.block_size);
        }
    }
}

// wc: weight * cos of this lane's 16 elements; ws: the weight of the other
// element of each pair * the sine with its sign in this one
template <bool INTER>
__device__ __forceinline__ void fold(const float* w, const float2* turn, int c0, int gap, bool turned0, bool turned1,
                                     uint64_t (&wc)[8], uint64_t (&ws)[8]) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {  // pairs of elements of both chunks
        float2 a = make_float2(1.f, 1.f), b = a;
        if (w != nullptr) {
            a = __ldg(reinterpret_cast<const float2*>(w + 8 * c0) + h);
            b = __ldg(reinterpret_cast<const float2*>(w + 8 * c0 + gap) + h);
        }
        if constexpr (INTER) {
            float2 f = turned0 ? turn[4 * c0 + h] : make_float2(1.f, 0.f);
            wc[h] = pair2(a.x * f.x, a.y * f.x);
            ws[h] = pair2(a.y * -f.y, a.x * f.y);
            f = turned1 ? turn[4 * c0 + gap / 2 + h] : make_float2(1.f, 0.f);
            wc[4 + h] = pair2(b.x * f.x, b.y * f.x);
            ws[4 + h] = pair2(b.y * -f.y, b.x * f.y);
        } else {
            float4 f = make_float4(1.f, 0.f, 1.f, 0.f);
            if (turned0) f = *reinterpret_cast<const float4*>(turn + 8 * c0 + 2 * h);
            wc[h] = pair2(a.x * f.x, a.y * f.z);
            ws[h] = pair2(b.x * -f.y, b.y * -f.w);
            wc[4 + h] = pair2(b.x * f.x, b.y * f.z);
            ws[4 + h] = pair2(a.x * f.y, a.y * f.w);
        }
    }
}

// Steps [s0, s0 + n) of the token's queries (KIND 0), keys (1) or values (2).
template <int DT, int KVT, int D, bool INTER, int KIND, bool NORM>
__device__ __forceinline__ void do_steps(const NormRopeParams& p, Run<KVT, D>& u, int s0, int n) {
    constexpr int LPR = D / 16, RPS = 32 / LPR;
    constexpr int ES = KIND != 0 && KVT == PA_FP8_E4M3 ? 1 : 2;  // bytes of an output element
    uint64_t wc[8], ws[8];
    if constexpr (KIND != 2) {
        work_out_sines(p, u);
        fold<INTER>(NORM ? (KIND == 0 ? p.q_weight : p.k_weight) : nullptr, u.turn, u.c0, u.gap, u.turned0, u.turned1,
                    wc, ws);
    }
    // this lane's first chunk of the output, and the way to the next step's
    uint8_t* dst;
    int64_t way;
    int rows = (KIND == 0 ? p.num_heads : p.num_kv_heads) - s0 * RPS - u.sub;
    const int64_t h0 = s0 * RPS + u.sub;
    if constexpr (KIND == 0) {
        dst = reinterpret_cast<uint8_t*>(p.q_out + u.tok.t * p.qo_stride + h0 * D + u.c0 * 8);
        way = RPS * D * 2;
    } else if constexpr (KVT == kPacked) {
        dst = reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(p.k_out) + u.tok.t * p.ko_stride + h0 * D + u.c0 * 8);
        way = RPS * D * 2;
    } else {
        dst = static_cast<uint8_t*>(KIND == 2 ? p.v_out : p.k_out) + ((u.at + h0 * p.block_size) * D + u.c0 * 8) * ES;
        way = static_cast<int64_t>(RPS) * p.block_size * D * ES;
        if (u.at < 0) rows = 0;  // no place: the rows are read and left
    }
    for (int i = 0; i < n; ++i, dst += way, rows -= RPS) {
        // all but the newest kDepth - 2 copies have landed: this step's among them
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
        const uint4 raw0 = u.ring[u.slot * 64], raw1 = u.ring[u.slot * 64 + 32];
        // the slot of the step before, whose row is used up, takes the next row
        u.load.issue(p, u.ring + (u.slot == 0 ? kDepth - 1 : u.slot - 1) * 64, u.sub, u.c0, u.gap);
        u.slot = u.slot == kDepth - 1 ? 0 : u.slot + 1;
        const uint32_t x[8] = {raw0.x, raw0.y, raw0.z, raw0.w, raw1.x, raw1.y, raw1.z, raw1.w};
        uint64_t y[8];
        if constexpr (KIND != 2 || ES == 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = widen<DT>(x[e]);
        }
        if constexpr (KIND != 2) {
            uint64_t r2 = 0;
            if constexpr (NORM) {
                uint64_t sa = mul2(y[0], y[0]), sb = mul2(y[4], y[4]);
#pragma unroll
                for (int e = 1; e < 4; ++e) {
                    sa = fma2(y[e], y[e], sa);
                    sb = fma2(y[4 + e], y[4 + e], sb);
                }
                const float2 s2 = unpair2(add2(sa, sb));
                float ss = s2.x + s2.y;
#pragma unroll
                for (int d = 1; d < LPR; d <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
                const float ms = fmaf(ss, 1.f / D, p.eps);
                float r = rsqrtf(ms);
                // squares, or a sum of squares and eps, past fp32's range on either
                // side (bf16 rows beyond 10^18; rows below 10^-15 with an eps as
                // small): again on the row scaled by a power of two, eps by its square
                const bool far = !(ms > 1.262177448e-29f && ms < INFINITY);  // 2^-96
                if (__any_sync(0xffffffffu, far)) {
                    const float by = !far ? 1.f : ms < 1.f ? 1.180591621e+21f : 8.470329473e-22f;  // 2^70, 2^-70
                    const uint64_t by2 = pair2(by, by);
                    float sd = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        y[e] = mul2(y[e], by2);
                        const float2 f = unpair2(y[e]);
                        sd = fmaf(f.x, f.x, fmaf(f.y, f.y, sd));
                    }
#pragma unroll
                    for (int d = 1; d < LPR; d <<= 1) sd += __shfl_xor_sync(0xffffffffu, sd, d);
                    if (far) r = rsqrtf(fmaf(sd, 1.f / D, p.eps * by * by));
                }
                r2 = pair2(r, r);
            }
            // an element that nothing turns takes no part of another (which may be infinite)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint64_t z0, z1;  // the other elements of the pairs
                if constexpr (INTER) {
                    const float2 f = unpair2(y[e]), g = unpair2(y[4 + e]);
                    z0 = pair2(f.y, f.x);
                    z1 = pair2(g.y, g.x);
                } else {
                    z0 = y[4 + e];
                    z1 = y[e];
                }
                y[e] = mul2(y[e], wc[e]);
                y[4 + e] = mul2(y[4 + e], wc[4 + e]);
                if (u.turned0) y[e] = fma2(z0, ws[e], y[e]);
                if (u.turned1) y[4 + e] = fma2(z1, ws[4 + e], y[4 + e]);
                if constexpr (NORM) {
                    y[e] = mul2(y[e], r2);
                    y[4 + e] = mul2(y[4 + e], r2);
                }
            }
        }
        if (rows <= 0) continue;
        if constexpr (ES == 1) {
            const float scale = KIND == 2 ? p.v_scale : p.k_scale;
            const float inverse = KIND == 2 ? p.v_inverse : p.k_inverse;
            *reinterpret_cast<uint2*>(dst) = e4m3_8(y, scale, inverse);
            *reinterpret_cast<uint2*>(dst + u.gap) = e4m3_8(y + 4, scale, inverse);
        } else {
            // (elements that nothing changed keep their bits)
            const bool vec = KIND == 0 ? p.qo_vec : KVT == kPacked ? p.ko_vec : true;
            const bool new0 = KIND != 2 && (NORM || u.turned0), new1 = KIND != 2 && (NORM || u.turned1);
            uint16_t* d16 = reinterpret_cast<uint16_t*>(dst);
            store_row8(d16, new0 ? round_8<DT>(y) : raw0, vec);
            store_row8(d16 + u.gap, new1 ? round_8<DT>(y + 4) : raw1, vec);
        }
    }
}

// DT: type of the rows; KVT: kPacked, DT (16-bit cache) or PA_FP8_E4M3
template <int DT, int KVT, int D, bool INTER>
__global__ void __launch_bounds__(kWarps * 32, kBlocks)
qk_norm_rope_kernel(const NormRopeParams p) {
    constexpr int LPR = D / 16;     // lanes per row, 16 elements each
    constexpr int RPS = 32 / LPR;   // rows of a step
    __shared__ __align__(16) float2 turn_all[kWarps][D / 2];
    __shared__ uint4 ring_all[kWarps][kDepth][2][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const int qs = (p.num_heads + RPS - 1) / RPS, ks = (p.num_kv_heads + RPS - 1) / RPS;
    const int steps = qs + ks * (KVT == kPacked ? 1 : 2);
    // the last run: the token, segment and step it begins at
    const int64_t begin = w * p.per_warp + (w < p.extra ? w : p.extra);
    const int64_t run = p.per_warp + (w < p.extra ? 1 : 0);
    int64_t left = p.rounds * steps + run;
    if (left == 0) return;
    Run<KVT, D> u;
    u.tok.last = p.rounds * p.warps + begin / steps;
    int i = static_cast<int>(begin % steps);
    u.load.first_seg = i < qs ? 0 : i < qs + ks ? 1 : 2;
    u.load.first_step = i - (i < qs ? 0 : i < qs + ks ? qs : qs + ks);
    u.tok.round = 0;
    u.tok.t = p.rounds > 0 ? w : u.tok.last;
    int seg = p.rounds > 0 ? 0 : u.load.first_seg;
    i = p.rounds > 0 ? 0 : u.load.first_step;
    u.ring = &ring_all[warp][0][0][lane];
    u.slot = 0;
    u.turn = turn_all[warp];
    u.sub = lane / LPR;
    u.half = p.rotary_dim / 16;
    const int j = lane % LPR;
    if (INTER) {
        u.c0 = j;
        u.gap = LPR * 8;
        u.turned0 = j < 2 * u.half;
        u.turned1 = j + LPR < 2 * u.half;
    } else {
        u.turned0 = u.turned1 = j < u.half;
        u.c0 = j < u.half ? j : j + u.half;
        u.gap = (j < u.half ? u.half : LPR - u.half) * 8;
    }
    u.at = -1;
    u.next_pos = u.half > 0 ? __ldg(p.positions + u.tok.t) : 0;
    u.next_slot = KVT != kPacked ? __ldg(p.slots + u.tok.t) : -1;
    u.load.at = u.tok;
    u.load.seg = seg;
    u.load.left = left;
    u.load.enter(p, i, u.sub, u.c0);
#pragma unroll
    for (int k = 0; k < kDepth - 1; ++k) u.load.issue(p, u.ring + k * 64, u.sub, u.c0, u.gap);
    enter_token(p, u);
    while (left > 0) {
        const int n = static_cast<int>(min(left, static_cast<int64_t>((seg == 0 ? qs : ks) - i)));
        if (seg == 0) {
            if (p.q_weight != nullptr) do_steps<DT, KVT, D, INTER, 0, true>(p, u, i, n);
            else do_steps<DT, KVT, D, INTER, 0, false>(p, u, i, n);
        } else if (seg == 1) {
            if (p.k_weight != nullptr) do_steps<DT, KVT, D, INTER, 1, true>(p, u, i, n);
            else do_steps<DT, KVT, D, INTER, 1, false>(p, u, i, n);
        } else if constexpr (KVT != kPacked) {
            do_steps<DT, KVT, D, INTER, 2, false>(p, u, i, n);
        }
        left -= n;
        i = 0;
        if (++seg == Loader<KVT, D>::kSegs && left > 0) {
            seg = 0;
            u.tok.next(p);
            if (u.tok.round == p.rounds) {
                seg = u.load.first_seg;
                i = u.load.first_step;
            }
            enter_token(p, u);
        }
    }
    // (the run's last groups are empty: no copy is on its way)
}

// 1 / x where x is a power of two (and 1 / x a normal number), else 0
float power_of_two_inverse(float x) {
    int e;
    return std::frexp(x, &e) == 0.5f && e >= -125 && e <= 126 ? 1.f / x : 0.f;
}

bool aligned16(const void* ptr, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0 && stride % 8 == 0;
}

template <int DT, int KVT, int D, bool INTER>
pa_status launch_t(NormRopeParams p, cudaStream_t stream) {
    constexpr int RPS = 512 / D;
    const int64_t sms = device_sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    const int ks = (p.num_kv_heads + RPS - 1) / RPS;
    const int steps = (p.num_heads + RPS - 1) / RPS + ks * (KVT == kPacked ? 1 : 2);
    static LaunchCache cache;
    const int per_sm = blocks_per_sm(qk_norm_rope_kernel<DT, KVT, D, INTER>, kWarps * 32, 0, cache);
    if (per_sm <= 0) return PA_ERR_CUDA;
    if (p.num_tokens > INT64_MAX / (1 << 20)) return PA_ERR_UNSUPPORTED;
    const int64_t total = p.num_tokens * steps;
    int64_t blocks = (total + kWarps - 1) / kWarps;  // a step a warp, at least
    if (blocks > sms * per_sm) blocks = sms * per_sm;
    p.warps = blocks * kWarps;
    p.rounds = p.num_tokens / p.warps;
    const int64_t rest = total - p.rounds * p.warps * steps;
    p.per_warp = rest / p.warps;
    p.extra = rest % p.warps;
    return launch_pdl(qk_norm_rope_kernel<DT, KVT, D, INTER>, static_cast<int>(blocks), kWarps * 32, 0, stream, p) ==
                   cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

pa_status launch(const NormRopeParams& p, int dt, int kvt, int head_size, cudaStream_t s) {
#define PA_CASE(DT, KVT, D) \
    if (dt == DT && kvt == KVT && head_size == D)  \
        return p.interleaved ? launch_t<DT, KVT, D, true>(p, s) : launch_t<DT, KVT, D, false>(p, s);
#define PA_TYPES(D)                                                                              \
    PA_CASE(PA_F16, kPacked, D) PA_CASE(PA_F16, PA_F16, D) PA_CASE(PA_F16, PA_FP8_E4M3, D)       \
    PA_CASE(PA_BF16, kPacked, D) PA_CASE(PA_BF16, PA_BF16, D) PA_CASE(PA_BF16, PA_FP8_E4M3, D)
    PA_TYPES(64)
    PA_TYPES(128)
#undef PA_TYPES
#undef PA_CASE
    return PA_ERR_UNSUPPORTED;
}

// what both entry points check; fills in the shared part of p
pa_status prepare(NormRopeParams& p, void* q_out, const void* q, const void* k, pa_dtype dtype, int64_t num_tokens,
                  int32_t num_heads, int32_t num_kv_heads, int32_t head_size, int64_t q_stride, int64_t k_stride,
                  int64_t q_out_stride, const int64_t* positions, const pa_qk_transform* tr) {
    if (tr == nullptr || num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0) return PA_ERR_INVALID_ARG;
    if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (head_size != 64 && head_size != 128) return PA_ERR_UNSUPPORTED;
    // (a row's index inside a tile, and a token's row offsets, are 32-bit)
    if (num_heads > 4096 || num_kv_heads > 4096) return PA_ERR_UNSUPPORTED;
    const int64_t qrow = static_cast<int64_t>(num_heads) * head_size;
    const int64_t krow = static_cast<int64_t>(num_kv_heads) * head_size;
    if (q_stride < qrow || q_out_stride < qrow || k_stride < krow) return PA_ERR_INVALID_ARG;
    if (tr->rotary_dim < 0 || tr->rotary_dim > head_size) return PA_ERR_INVALID_ARG;
    if (tr->rotary_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
    if (tr->rotary_dim > 0 && (tr->turns == nullptr || (reinterpret_cast<uintptr_t>(tr->turns) & 7u) ||
                               !std::isfinite(tr->rope_factor)))
        return PA_ERR_INVALID_ARG;
    if ((tr->q_weight != nullptr || tr->k_weight != nullptr) && !(tr->eps > 0.f && std::isfinite(tr->eps)))
        return PA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(tr->q_weight) & 15u) || (reinterpret_cast<uintptr_t>(tr->k_weight) & 15u))
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (q_out == nullptr || q == nullptr || k == nullptr || (tr->rotary_dim > 0 && positions == nullptr))
        return PA_ERR_INVALID_ARG;
    // in place, a token's rows have to stay where they are
    if (q_out == q && q_out_stride != q_stride && num_tokens > 1) return PA_ERR_INVALID_ARG;
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.q_out = static_cast<uint16_t*>(q_out);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.qo_stride = q_out_stride;
    p.positions = positions;
    p.turns = tr->turns;
    p.q_weight = tr->q_weight;
    p.k_weight = tr->k_weight;
    p.num_tokens = num_tokens;
    p.eps = tr->eps;
    p.rope_factor = tr->rope_factor;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.rotary_dim = tr->rotary_dim;
    p.interleaved = tr->interleaved != 0 ? 1 : 0;
    p.q_vec = aligned16(q, q_stride);
    p.k_vec = aligned16(k, k_stride);
    p.qo_vec = aligned16(q_out, q_out_stride);
    return PA_OK;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_qk_norm_rope(void* q_out, void* k_out, const void* q, const void* k, pa_dtype dtype,
                                     int64_t num_tokens, int32_t num_heads, int32_t num_kv_heads, int32_t head_size,
                                     int64_t q_stride, int64_t k_stride, int64_t q_out_stride, int64_t k_out_stride,
                                     const int64_t* positions, const pa_qk_transform* transform,
                                     pa_stream_t stream) {
    NormRopeParams p{};
    const pa_status st = prepare(p, q_out, q, k, dtype, num_tokens, num_heads, num_kv_heads, head_size, q_stride,
                                 k_stride, q_out_stride, positions, transform);
    if (st != PA_OK) return st;
    if (k_out_stride < static_cast<int64_t>(num_kv_heads) * head_size) return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (k_out == nullptr || (k_out == k && k_out_stride != k_stride && num_tokens > 1)) return PA_ERR_INVALID_ARG;
    p.k_out = k_out;
    p.ko_stride = k_out_stride;
    p.ko_vec = aligned16(k_out, k_out_stride);
    return launch(p, dtype, kPacked, head_size, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" pa_status pa_qk_norm_rope_write(void* q_out, const void* q, const void* k, const void* v, pa_dtype dtype,
                                           const pa_kv_cache* cache, int64_t num_tokens, int32_t num_heads,
                                           int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                           int64_t q_out_stride, const int64_t* positions,
                                           const int64_t* slot_mapping, const pa_qk_transform* transform,
                                           int32_t* dev_status, pa_stream_t stream) {
    pa_status st = check_cache(cache);
    if (st != PA_OK) return st;
    NormRopeParams p{};
    st = prepare(p, q_out, q, k, dtype, num_tokens, num_heads, cache->num_kv_heads, cache->head_size, q_stride,
                 k_stride, q_out_stride, positions, transform);
    if (st != PA_OK) return st;
    if (v_stride < static_cast<int64_t>(cache->num_kv_heads) * cache->head_size) return PA_ERR_INVALID_ARG;
    const bool fp8 = cache->kv_dtype == PA_FP8_E4M3;
    if (!fp8 && cache->kv_dtype != dtype) return PA_ERR_UNSUPPORTED;
    if (fp8 && !(cache->k_scale > 0.f && std::isfinite(cache->k_scale) && cache->v_scale > 0.f &&
                 std::isfinite(cache->v_scale)))
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (v == nullptr || slot_mapping == nullptr) return PA_ERR_INVALID_ARG;
    p.v = static_cast<const uint16_t*>(v);
    p.v_stride = v_stride;
    p.v_vec = aligned16(v, v_stride);
    p.k_out = cache->k_cache;
    p.v_out = cache->v_cache;
    p.slots = slot_mapping;
    p.status = dev_status;
    p.block_size = cache->block_size;
    p.num_slots = cache->num_blocks * cache->block_size;
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    p.k_inverse = power_of_two_inverse(cache->k_scale);
    p.v_inverse = power_of_two_inverse(cache->v_scale);
    return launch(p, dtype, fp8 ? PA_FP8_E4M3 : static_cast<int>(dtype), cache->head_size,
                  reinterpret_cast<cudaStream_t>(stream));
}
