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
// The kernel is bandwidth-bound: 2 bytes in and 2 (or 1) out per element
// against about 10 instructions.  A row is handled by D/8 lanes, one 16-byte
// load and store each, so a warp takes 2 or 4 heads at a time; a warp's unit is
// one token, or part of its rows when there are few tokens.  Per unit the warp
// works out the token's sines (two per lane, exchanged through shared memory)
// while its first rows are in flight, and folds the norm's weights into them:
//     out = r (x w cos + x' w' sin),  r = 1 / sqrt(mean(x^2) + eps),
// with x' the other element of the pair, which is swapped between lanes as the
// 16-bit input it came as.
#include <cmath>

#include "common.cuh"
#include "launch.h"

namespace pa {
namespace {

constexpr int kWarps = 4;        // units of a block, one a warp
constexpr int kUnroll = 4;       // rows a lane loads before it works on the first
constexpr int kBlocks = 6;       // blocks per SM that the registers allow
constexpr int kUnitsPerSm = 96;  // units wanted per SM
constexpr int kMinSteps = 2;     // steps of a unit, at least, when a token is split
constexpr int kPacked = -1;      // keys go to packed rows, there is no cache

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
    int32_t num_heads, num_kv_heads;
    int32_t rotary_dim, interleaved, block_size;
    int32_t parts;     // units of a token
    int32_t per_part;  // steps of a unit (a step: the rows a warp takes at a time)
    // 16-byte accesses allowed (pointer and stride aligned)
    bool q_vec, k_vec, v_vec, qo_vec, ko_vec;
};

__device__ __forceinline__ uint4 load_row8(const uint16_t* p, bool vec) {
    if (vec) return __ldcs(reinterpret_cast<const uint4*>(p));
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

// 8 values -> 8 E4M3 codes: IEEE division, then one rounding with saturation
__device__ __forceinline__ uint2 e4m3_8(const float (&x)[8], float scale) {
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c[j] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
            make_float2(__fdiv_rn(x[2 * j], scale), __fdiv_rn(x[2 * j + 1], scale)), __NV_SATFINITE, __NV_E4M3));
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
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
template <int DT>
__device__ __forceinline__ uint64_t widen(uint32_t w) {
    const float2 f = kv_pair<DT>(w);
    return pair2(f.x, f.y);
}

// The state of a warp's unit: its token, this lane's place in the rows, the
// sines once they are worked out.
struct Unit {
    int64_t t;     // token
    int64_t at;    // cache row of the token's KV head 0, -1 for none
    float2* turn;  // shared memory: (cos, sin) * factor of the token's pairs
    int c, sub;    // chunk of 8 elements, row of a step
    int half;      // chunks of half the rotated part
    int other;     // half layout: chunk that holds the other elements of this lane's pairs
    bool rotated;
    bool ready;  // the sines are in `turn`
};

__device__ __forceinline__ void work_out_sines(const NormRopeParams& p, Unit& u) {
    if (u.ready || u.half == 0) return;
    u.ready = true;
    const uint64_t pos = static_cast<uint64_t>(__ldg(p.positions + u.t));
    for (int i = threadIdx.x & 31; i < p.rotary_dim / 2; i += 32) {
        // the signed top half of the phase is the fraction of a turn in units
        // of 2^-32, so * 2^-31 gives half turns in [-1, 1)
        const int32_t frac = static_cast<int32_t>((pos * __ldg(p.turns + i)) >> 32);
        float s, c;
        sincospif(static_cast<float>(frac) * 4.656612873077393e-10f, &s, &c);
        u.turn[i] = make_float2(c * p.rope_factor, s * p.rope_factor);
    }
    __syncwarp();
}

// Steps [s0, s1) of the token's queries (KIND 0), keys (1) or values (2).
template <int DT, int KVT, int D, int KIND>
__device__ __forceinline__ void do_steps(const NormRopeParams& p, Unit& u, int s0, int s1) {
    constexpr int LPR = D / 8, RPS = 32 / LPR;
    if (s0 >= s1) return;
    const int n = KIND == 0 ? p.num_heads : p.num_kv_heads;
    const uint16_t* src = (KIND == 0 ? p.q + u.t * p.q_stride : KIND == 1 ? p.k + u.t * p.k_stride
                                                                          : p.v + u.t * p.v_stride) + u.c * 8;
    const bool vec = KIND == 0 ? p.q_vec : KIND == 1 ? p.k_vec : p.v_vec;
    const float* w = KIND == 0 ? p.q_weight : p.k_weight;
    const bool norm = KIND != 2 && w != nullptr;
    const int partner = (threadIdx.x & 31 & ~(LPR - 1)) + u.other;
    uint64_t wc[4], ws[4];  // weight * cos, the other element's weight * signed sin
    for (int i = s0; i < s1; i += kUnroll) {
        uint4 raw[kUnroll];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int h = (i + j) * RPS + u.sub;
            raw[j] = i + j < s1 && h < n ? load_row8(src + h * D, vec) : make_uint4(0u, 0u, 0u, 0u);
        }
        if (KIND != 2 && i == s0) {
            work_out_sines(p, u);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float2 a = make_float2(1.f, 1.f), b = a, f0 = make_float2(1.f, 0.f), f1 = f0;
                if (norm) {
                    a = __ldg(reinterpret_cast<const float2*>(w) + 4 * u.c + e);
                    b = p.interleaved ? make_float2(a.y, a.x)
                                      : __ldg(reinterpret_cast<const float2*>(w) + 4 * u.other + e);
                }
                if (u.rotated) {
                    if (p.interleaved) {
                        f1 = u.turn[4 * u.c + e];
                        f0 = make_float2(f1.x, -f1.y);
                    } else {
                        const bool low = u.c < u.half;
                        const float4 f = *reinterpret_cast<const float4*>(u.turn + 8 * (low ? u.c : u.c - u.half) + 2 * e);
                        f0 = make_float2(f.x, low ? -f.y : f.y);
                        f1 = make_float2(f.z, low ? -f.w : f.w);
                    }
                }
                wc[e] = pair2(a.x * f0.x, a.y * f1.x);
                ws[e] = pair2(b.x * f0.y, b.y * f1.y);
            }
        }
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            if (i + j >= s1) break;
            uint32_t x[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
            uint64_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = widen<DT>(x[e]);
            if constexpr (KIND != 2) {
                uint64_t z[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    z[e] = widen<DT>(p.interleaved ? __byte_perm(x[e], 0u, 0x1032)
                                                   : __shfl_sync(0xffffffffu, x[e], partner));
                float r = 1.f;
                if (norm) {
                    uint64_t s2 = mul2(o[0], o[0]);
#pragma unroll
                    for (int e = 1; e < 4; ++e) s2 = fma2(o[e], o[e], s2);
                    const float2 sp = unpair2(s2);
                    float ss = sp.x + sp.y;
#pragma unroll
                    for (int d = 1; d < LPR; d <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
                    r = rsqrtf(fmaf(ss, 1.f / D, p.eps));
                    // squares past fp32's range (bf16 rows beyond 10^18): again
                    // on the row scaled by 2^-70, next to which eps is nothing
                    const bool big = !(ss < INFINITY);
                    if (__any_sync(0xffffffffu, big)) {
                        const float down = big ? 8.470329472543003e-22f : 1.f;
                        const uint64_t d2 = pair2(down, down);
                        float sb = 0.f;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            o[e] = mul2(o[e], d2);
                            z[e] = mul2(z[e], d2);
                            const float2 f = unpair2(o[e]);
                            sb = fmaf(f.x, f.x, fmaf(f.y, f.y, sb));
                        }
#pragma unroll
                        for (int d = 1; d < LPR; d <<= 1) sb += __shfl_xor_sync(0xffffffffu, sb, d);
                        if (big) r = rsqrtf(sb * (1.f / D));
                    }
                }
                const uint64_t r2 = pair2(r, r);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // an element that nothing turns takes no part of another (which may be infinite)
                    o[e] = mul2(o[e], wc[e]);
                    if (u.rotated) o[e] = fma2(z[e], ws[e], o[e]);
                    if (norm) o[e] = mul2(o[e], r2);
                }
            }
            const int h = (i + j) * RPS + u.sub;
            if (h >= n) continue;
            uint4 out = raw[j];
            // (elements that nothing changed keep their bits)
            if (KIND != 2 && (norm || u.rotated)) {
                uint32_t y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpair2(o[e]);
                    y[e] = round_pair<DT>(f.x, f.y);
                }
                out = make_uint4(y[0], y[1], y[2], y[3]);
            }
            if constexpr (KIND == 0) {
                store_row8(p.q_out + u.t * p.qo_stride + h * D + u.c * 8, out, p.qo_vec);
            } else if constexpr (KVT == kPacked) {
                store_row8(static_cast<uint16_t*>(p.k_out) + u.t * p.ko_stride + h * D + u.c * 8, out, p.ko_vec);
            } else if (u.at >= 0) {
                const int64_t off = (u.at + static_cast<int64_t>(h) * p.block_size) * D + u.c * 8;
                void* dst = KIND == 2 ? p.v_out : p.k_out;
                if constexpr (KVT == PA_FP8_E4M3) {
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 g = unpair2(o[e]);
                        f[2 * e] = g.x;
                        f[2 * e + 1] = g.y;
                    }
                    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(dst) + off) =
                        e4m3_8(f, KIND == 2 ? p.v_scale : p.k_scale);
                } else {
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + off) = out;
                }
            }
        }
    }
}

// DT: type of the rows; KVT: kPacked, DT (16-bit cache) or PA_FP8_E4M3
template <int DT, int KVT, int D>
__global__ void __launch_bounds__(kWarps * 32, kBlocks)
qk_norm_rope_kernel(const NormRopeParams p) {
    constexpr int LPR = D / 8;      // lanes per row, 8 elements each
    constexpr int RPS = 32 / LPR;   // rows of a step
    __shared__ __align__(16) float2 turn_all[kWarps][D / 2];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (unit >= p.num_tokens * p.parts) return;
    Unit u;
    u.t = p.parts == 1 ? unit : unit / p.parts;
    u.turn = turn_all[warp];
    u.c = lane % LPR;
    u.sub = lane / LPR;
    u.half = p.rotary_dim / 16;
    u.rotated = u.c < 2 * u.half;
    u.other = p.interleaved || !u.rotated ? u.c : (u.c < u.half ? u.c + u.half : u.c - u.half);
    u.ready = false;
    u.at = -1;

    // the token's steps: queries, keys, values; this unit takes [i0, i1)
    const int qs = (p.num_heads + RPS - 1) / RPS, ks = (p.num_kv_heads + RPS - 1) / RPS;
    const int i0 = static_cast<int>(unit - u.t * p.parts) * p.per_part, i1 = i0 + p.per_part;
    if (KVT != kPacked && i1 > qs) {
        const int64_t slot = __ldg(p.slots + u.t);
        if (slot >= p.num_slots) {
            if (lane == 0) report(p.status, PA_ERR_BAD_BLOCK);
        } else if (slot >= 0) {
            // (a 32-bit division where it does: a 64-bit one is ten times as long)
            const int64_t blk = slot >> 32 == 0 ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.block_size)
                                                : slot / p.block_size;
            u.at = blk * p.num_kv_heads * p.block_size + (slot - blk * p.block_size);
        }
    }
    do_steps<DT, KVT, D, 0>(p, u, i0, min(i1, qs));
    do_steps<DT, KVT, D, 1>(p, u, max(i0 - qs, 0), min(i1 - qs, ks));
    if constexpr (KVT != kPacked) do_steps<DT, KVT, D, 2>(p, u, max(i0 - qs - ks, 0), min(i1 - qs - ks, ks));
}

bool aligned16(const void* ptr, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0 && stride % 8 == 0;
}

template <int DT, int KVT, int D>
pa_status launch_t(NormRopeParams p, cudaStream_t stream) {
    constexpr int RPS = 32 / (D / 8);
    const int64_t sms = device_sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    const int ks = (p.num_kv_heads + RPS - 1) / RPS;
    const int steps = (p.num_heads + RPS - 1) / RPS + ks * (KVT == kPacked ? 1 : 2);
    // units of a token: one (its sines are worked out once), more while the
    // units would not fill the SMs' warps a few times over
    const int64_t want = sms * kUnitsPerSm / p.num_tokens;
    const int64_t most = (steps + kMinSteps - 1) / kMinSteps;
    const int parts = static_cast<int>(want < 1 ? 1 : (want < most ? want : most));
    p.per_part = (steps + parts - 1) / parts;
    p.parts = (steps + p.per_part - 1) / p.per_part;
    const int64_t blocks = (p.num_tokens * p.parts + kWarps - 1) / kWarps;
    if (blocks > INT32_MAX) return PA_ERR_UNSUPPORTED;
    return launch_pdl(qk_norm_rope_kernel<DT, KVT, D>, static_cast<int>(blocks), kWarps * 32, 0, stream, p) ==
                   cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

pa_status launch(const NormRopeParams& p, int dt, int kvt, int head_size, cudaStream_t s) {
#define PA_CASE(DT, KVT, D) \
    if (dt == DT && kvt == KVT && head_size == D) return launch_t<DT, KVT, D>(p, s);
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
    if (tr->rotary_dim > 0 && (tr->turns == nullptr || !std::isfinite(tr->rope_factor))) return PA_ERR_INVALID_ARG;
    if ((tr->q_weight != nullptr || tr->k_weight != nullptr) && !(tr->eps > 0.f && std::isfinite(tr->eps)))
        return PA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(tr->q_weight) & 15u) || (reinterpret_cast<uintptr_t>(tr->k_weight) & 15u))
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (q_out == nullptr || q == nullptr || k == nullptr || (tr->rotary_dim > 0 && positions == nullptr))
        return PA_ERR_INVALID_ARG;
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
    if (k_out == nullptr) return PA_ERR_INVALID_ARG;
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
    return launch(p, dtype, fp8 ? PA_FP8_E4M3 : static_cast<int>(dtype), cache->head_size,
                  reinterpret_cast<cudaStream_t>(stream));
}
