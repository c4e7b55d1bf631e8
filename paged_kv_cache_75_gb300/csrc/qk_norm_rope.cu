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
// against about 10 instructions.  A row is handled by D/8 lanes with one 16-byte
// load and store each; a block of 256 threads takes a few tokens (all of their
// rows), so each token's sines are worked out once per block, in shared memory,
// while its rows' loads are in flight.
#include <cmath>

#include "common.cuh"
#include "launch.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;       // rows a lane group loads before it works on the first
constexpr int kMaxTokens = 32;   // tokens of a block's tile
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
    int32_t num_heads, num_kv_heads, rows;  // rows of a token: H + Hkv (+ Hkv values)
    int32_t rotary_dim, interleaved, block_size;
    int32_t tile;    // tokens of a block's tile
    int32_t splits;  // blocks that share a one-token tile's rows
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

// DT: type of the rows; KVT: kPacked, DT (16-bit cache) or PA_FP8_E4M3
template <int DT, int KVT, int D>
__global__ void __launch_bounds__(kThreads)
qk_norm_rope_kernel(const NormRopeParams p) {
    constexpr int LPR = D / 8;               // lanes per row, 8 elements each
    constexpr int GROUPS = kThreads / LPR;   // rows in work at a time
    __shared__ float2 turn[kMaxTokens][D / 2];  // (cos, sin) * factor of each token and pair
    __shared__ int64_t cache_row[kMaxTokens];   // row of KV head 0 in the cache, -1: none
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int c = threadIdx.x % LPR;   // this lane's 8-element chunk of its rows
    const int group = threadIdx.x / LPR;
    const int half = p.rotary_dim / 16;  // chunks of half the rotated part
    // half layout: the lane that holds the other element of this lane's pairs
    const bool rotated = c < 2 * half;
    const int partner = (lane & ~(LPR - 1)) + (!rotated ? c : c < half ? c + half : c - half);
    const int pair0 = p.interleaved ? 4 * c : 8 * (c < half ? c : c - half);
    const float side = c < half ? -1.f : 1.f;  // half layout: sign of the sine's term

    const int64_t tiles = (p.num_tokens + p.tile - 1) / p.tile;
    for (int64_t u = blockIdx.x; u < tiles * p.splits; u += gridDim.x) {
        const int64_t t0 = u / p.splits * p.tile;
        const int nt = static_cast<int>(min(static_cast<int64_t>(p.tile), p.num_tokens - t0));
        // rows [r0, r1) of the tile, token-major
        const int part = static_cast<int>(u % p.splits);
        const int r0 = part * GROUPS, step = p.splits * GROUPS, r1 = nt * p.rows;
        bool first = true;
        for (int base = r0; base < r1; base += step * kUnroll) {
            uint4 raw[kUnroll];
            int tok[kUnroll], row[kUnroll];
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) {
                const int rr = base + j * step + group;
                tok[j] = rr < r1 ? (nt == 1 ? 0 : rr / p.rows) : -1;
                row[j] = rr - tok[j] * p.rows;
                raw[j] = make_uint4(0u, 0u, 0u, 0u);
                if (tok[j] >= 0) {
                    const int64_t t = t0 + tok[j];
                    const int h = row[j];
                    if (h < p.num_heads)
                        raw[j] = load_row8(p.q + t * p.q_stride + h * D + c * 8, p.q_vec);
                    else if (h < p.num_heads + p.num_kv_heads)
                        raw[j] = load_row8(p.k + t * p.k_stride + (h - p.num_heads) * D + c * 8, p.k_vec);
                    else
                        raw[j] = load_row8(p.v + t * p.v_stride + (h - p.num_heads - p.num_kv_heads) * D + c * 8,
                                           p.v_vec);
                }
            }
            if (first) {
                first = false;
                const int pairs = p.rotary_dim / 2;
                for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
                    const int tt = nt == 1 ? 0 : i / pairs, pr = i - tt * pairs;
                    const uint64_t phase = static_cast<uint64_t>(__ldg(p.positions + t0 + tt)) * __ldg(p.turns + pr);
                    // the signed top half is the fraction of a turn in units of
                    // 2^-32, so * 2^-31 gives half turns in [-1, 1)
                    const float x = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f;
                    float s, co;
                    sincospif(x, &s, &co);
                    turn[tt][pr] = make_float2(co * p.rope_factor, s * p.rope_factor);
                }
                if constexpr (KVT != kPacked) {
                    if (threadIdx.x < nt) {
                        const int64_t slot = __ldg(p.slots + t0 + threadIdx.x);
                        int64_t at = -1;
                        if (slot >= p.num_slots) {
                            report(p.status, PA_ERR_BAD_BLOCK);
                        } else if (slot >= 0) {
                            const int64_t blk = slot / p.block_size;
                            at = blk * p.num_kv_heads * p.block_size + (slot - blk * p.block_size);
                        }
                        cache_row[threadIdx.x] = at;
                    }
                }
                __syncthreads();
            }
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) {
                const bool is_q = row[j] < p.num_heads;
                const bool is_v = row[j] >= p.num_heads + p.num_kv_heads;
                const int tt = tok[j] < 0 ? 0 : tok[j];
                const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
                float y[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = kv_pair<DT>(w[e]);
                    y[2 * e] = f.x;
                    y[2 * e + 1] = f.y;
                }
                const float* wt = is_q ? p.q_weight : p.k_weight;
                if (p.q_weight != nullptr || p.k_weight != nullptr) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
                    for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    float r = rsqrtf(fmaf(ss, 1.f / D, p.eps));
                    // squares past fp32's range (bf16 rows beyond 10^18): again
                    // on the row scaled by 2^-70, next to which eps is nothing
                    const bool big = !(ss < INFINITY);
                    if (__any_sync(0xffffffffu, big)) {
                        const float down = big ? 8.470329472543003e-22f : 1.f;
                        float s2 = 0.f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) s2 = fmaf(y[e] * down, y[e] * down, s2);
#pragma unroll
                        for (int o = 1; o < LPR; o <<= 1) s2 += __shfl_xor_sync(0xffffffffu, s2, o);
                        if (big) {
                            r = rsqrtf(s2 * (1.f / D));
                            if (wt != nullptr && !is_v) {
#pragma unroll
                                for (int e = 0; e < 8; ++e) y[e] *= down;
                            }
                        }
                    }
                    if (wt != nullptr && !is_v) {
                        const float4 w0 = __ldg(reinterpret_cast<const float4*>(wt) + 2 * c);
                        const float4 w1 = __ldg(reinterpret_cast<const float4*>(wt) + 2 * c + 1);
                        y[0] *= r * w0.x; y[1] *= r * w0.y; y[2] *= r * w0.z; y[3] *= r * w0.w;
                        y[4] *= r * w1.x; y[5] *= r * w1.y; y[6] *= r * w1.z; y[7] *= r * w1.w;
                    }
                }
                if (p.interleaved) {
                    if (rotated && !is_v) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 t = turn[tt][pair0 + e];
                            const float a = y[2 * e], b = y[2 * e + 1];
                            y[2 * e] = fmaf(a, t.x, -(b * t.y));
                            y[2 * e + 1] = fmaf(b, t.x, a * t.y);
                        }
                    }
                } else if (half > 0) {
                    float z[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[e] = __shfl_sync(0xffffffffu, y[e], partner);
                    if (rotated && !is_v) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float2 t = turn[tt][pair0 + e];
                            y[e] = fmaf(y[e], t.x, side * (z[e] * t.y));
                        }
                    }
                }
                if (tok[j] < 0) continue;
                const int64_t t = t0 + tok[j];
                // values, and rows that nothing changed, keep their bits
                const bool same = is_v || (wt == nullptr && !rotated);
                uint4 x = raw[j];
                if (!same)
                    x = make_uint4(round_pair<DT>(y[0], y[1]), round_pair<DT>(y[2], y[3]), round_pair<DT>(y[4], y[5]),
                                   round_pair<DT>(y[6], y[7]));
                if (is_q) {
                    store_row8(p.q_out + t * p.qo_stride + row[j] * D + c * 8, x, p.qo_vec);
                    continue;
                }
                const int h = row[j] - p.num_heads - (is_v ? p.num_kv_heads : 0);
                if constexpr (KVT == kPacked) {
                    store_row8(static_cast<uint16_t*>(p.k_out) + t * p.ko_stride + h * D + c * 8, x, p.ko_vec);
                } else {
                    const int64_t at = cache_row[tt];
                    if (at < 0) continue;
                    const int64_t off = (at + static_cast<int64_t>(h) * p.block_size) * D + c * 8;
                    void* dst = is_v ? p.v_out : p.k_out;
                    if constexpr (KVT == PA_FP8_E4M3)
                        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(dst) + off) =
                            e4m3_8(y, is_v ? p.v_scale : p.k_scale);
                    else
                        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + off) = x;
                }
            }
        }
        __syncthreads();  // the next tile writes the sines again
    }
}

bool aligned16(const void* ptr, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0 && stride % 8 == 0;
}

template <int DT, int KVT, int D>
pa_status launch_t(NormRopeParams p, cudaStream_t stream) {
    constexpr int GROUPS = kThreads / (D / 8);
    const int64_t sms = device_sm_count();
    if (sms <= 0) return PA_ERR_CUDA;
    // a tile of about kUnroll rows per lane group; fewer tokens when they would
    // leave SMs without a tile, and a token's rows over several blocks when
    // there are fewer tokens than SMs
    int64_t tile = GROUPS * kUnroll / p.rows;
    if (tile > p.num_tokens / sms) tile = p.num_tokens / sms;
    p.tile = static_cast<int32_t>(tile < 1 ? 1 : (tile > kMaxTokens ? kMaxTokens : tile));
    const int64_t most = (p.rows + GROUPS - 1) / GROUPS;
    p.splits = 1;
    if (p.tile == 1 && p.num_tokens < sms) {
        const int64_t want = sms / p.num_tokens;
        p.splits = static_cast<int32_t>(want < most ? want : most);
    }
    const int64_t units = (p.num_tokens + p.tile - 1) / p.tile * p.splits;
    const int grid = static_cast<int>(units < INT32_MAX ? units : INT32_MAX);
    return launch_pdl(qk_norm_rope_kernel<DT, KVT, D>, grid, kThreads, 0, stream, p) == cudaSuccess ? PA_OK
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
    p.rows = num_heads + num_kv_heads;
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
    p.rows = num_heads + 2 * cache->num_kv_heads;
    return launch(p, dtype, fp8 ? PA_FP8_E4M3 : static_cast<int>(dtype), cache->head_size,
                  reinterpret_cast<cudaStream_t>(stream));
}
