// Reordering of beam search (pa_beam_reorder): the block tables, lengths and slots of
// the beams that go on, and copies of the blocks that two of them would write into.
//
// "Как работает paged attention? (детально)" 3.3: the beams of a request refer to the
// same physical blocks and a shared block is copied before a sequence writes into it.
// New row i goes on from parent p with the token at position L = lens[p].  Every whole
// block stays shared, so reordering moves table rows, not the cache; only the partly
// filled block that holds position L must be one row's own: the first of a parent's
// children keeps it, the others get a spare block with its L % block_size rows.
//
// Bound by memory: 2 * L % bs rows of every KV head and layer per copied block, 16 bytes
// a thread (64 requests of four beams, 16 layers, 100 MB: 19.8 us, 5.2 TB/s; the first step
// of 48 requests in an E4M3 cache of four layers 12.6).  One launch does the tables (blocks with blockIdx.y = 0) and all layers' copies
// (a block a row and layer); each block finds for itself, from the parents alone, whether
// its row is a first child.
#include "common.cuh"
#include "launch.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kLayers = 96;  // layers a launch takes (their addresses are kernel parameters)

struct ReorderParams {
    const int32_t* parents;
    const int32_t* table_in;
    const int32_t* lens_in;
    const int32_t* spare;
    int32_t* table_out;
    int32_t* lens_out;
    int64_t* slots_out;
    int32_t* used_out;
    int32_t* status;
    int64_t num_blocks;
    int32_t num_rows;
    int32_t num_rows_in;
    int32_t max_blocks;
    int32_t block_size;
    int32_t num_kv_heads;
    int32_t row_bytes;  // of a token's row of one KV head
    int32_t tables;     // blockIdx.y = 0 writes the tables, layer y - 1 otherwise; else layer y
    void* k[kLayers];
    void* v[kLayers];
};

template <typename T>
__global__ void __launch_bounds__(kThreads)
beam_reorder_kernel(const __grid_constant__ ReorderParams p) {
    pdl_wait();
    pdl_trigger();
    const int i = blockIdx.x, t = threadIdx.x;
    const bool tables = p.tables && blockIdx.y == 0;
    const int layer = static_cast<int>(blockIdx.y) - p.tables;
    int parent = p.parents[i];
    int length = 0;
    if (parent >= p.num_rows_in) {
        if (tables && t == 0) report(p.status, PA_ERR_INVALID_ARG);
        parent = -1;
    }
    if (parent >= 0) {
        length = p.lens_in[parent];
        if (length < 0 || length >= static_cast<int64_t>(p.max_blocks) * p.block_size) {
            if (tables && t == 0) report(p.status, PA_ERR_INVALID_ARG);
            parent = -1;
        }
    }
    const int last = length / p.block_size, rest = length - last * p.block_size;
    if (!tables && (parent < 0 || rest == 0)) return;
    // an earlier row goes on from the same parent: its block is not this row's
    bool again = false;
    for (int j = t; j < i && parent >= 0; j += kThreads) again |= p.parents[j] == parent;
    again = __syncthreads_or(again);
    const bool fresh = parent >= 0 && (rest == 0 || again);
    const int32_t* src = p.table_in + static_cast<int64_t>(parent < 0 ? 0 : parent) * p.max_blocks;
    if (tables) {
        int32_t* dst = p.table_out + static_cast<int64_t>(i) * p.max_blocks;
        const int have = parent < 0 ? 0 : last + (rest > 0);
        int own = -1;
        if (parent >= 0) {
            own = fresh ? p.spare[i] : src[last];
            const bool good = own >= 0 && own < p.num_blocks;
            if (!good) own = -1;
            if (t == 0 && !good) report(p.status, PA_ERR_BAD_BLOCK);
        }
        for (int j = t; j < p.max_blocks; j += kThreads)
            dst[j] = parent >= 0 && j == last ? own : j < have ? src[j] : -1;
        if (t == 0) {
            p.lens_out[i] = parent < 0 ? 0 : length + 1;
            p.slots_out[i] = own < 0 ? -1 : static_cast<int64_t>(own) * p.block_size + rest;
            p.used_out[i] = fresh;
        }
        return;
    }
    if (!again) return;
    const int from = src[last], to = p.spare[i];
    if (from < 0 || from >= p.num_blocks || to < 0 || to >= p.num_blocks) {
        if (t == 0) report(p.status, PA_ERR_BAD_BLOCK);
        return;
    }
    // the first `rest` rows of each KV head's page, one run
    const int run = rest * p.row_bytes / static_cast<int>(sizeof(T));
    const int64_t page = static_cast<int64_t>(p.block_size) * p.row_bytes / static_cast<int64_t>(sizeof(T));
    const int n = run * p.num_kv_heads;
    const int64_t a = from * page * p.num_kv_heads, b = to * page * p.num_kv_heads;
    T* k = static_cast<T*>(p.k[layer]);
    T* v = static_cast<T*>(p.v[layer]);
    for (int x = t; x < n; x += kThreads) {
        const int h = x / run;
        const int64_t at = h * page + (x - h * run);
        const T kx = k[a + at], vx = v[a + at];
        k[b + at] = kx;
        v[b + at] = vx;
    }
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_beam_reorder(const pa_kv_cache* caches, int32_t num_layers, const int32_t* parents,
                                     int32_t num_rows, const int32_t* block_table, int32_t num_rows_in,
                                     int32_t max_blocks_per_seq, const int32_t* seq_lens, const int32_t* spare_blocks,
                                     int32_t* block_table_out, int32_t* seq_lens_out, int64_t* slot_mapping_out,
                                     int32_t* spare_used_out, int32_t* dev_status, pa_stream_t stream) {
    if (num_layers <= 0 || caches == nullptr || num_rows < 0 || num_rows_in < 0 || max_blocks_per_seq <= 0)
        return PA_ERR_INVALID_ARG;
    const pa_kv_cache& c = caches[0];
    for (int l = 0; l < num_layers; ++l) {
        const pa_status st = check_cache(caches + l);
        if (st != PA_OK) return st;
        const pa_kv_cache& x = caches[l];
        if (x.num_blocks != c.num_blocks || x.block_size != c.block_size || x.num_kv_heads != c.num_kv_heads ||
            x.head_size != c.head_size || x.kv_dtype != c.kv_dtype)
            return PA_ERR_INVALID_ARG;
    }
    if (num_rows == 0) return PA_OK;
    if (parents == nullptr || spare_blocks == nullptr || block_table_out == nullptr || seq_lens_out == nullptr ||
        slot_mapping_out == nullptr || spare_used_out == nullptr)
        return PA_ERR_INVALID_ARG;
    if (num_rows_in > 0 && (block_table == nullptr || seq_lens == nullptr)) return PA_ERR_INVALID_ARG;
    // new rows overwrite what other rows still have to read
    if (block_table_out == block_table || seq_lens_out == seq_lens) return PA_ERR_INVALID_ARG;
    const int64_t row_bytes = static_cast<int64_t>(c.head_size) * elem_bytes(c.kv_dtype);
    if (row_bytes * c.block_size * c.num_kv_heads > INT32_MAX) return PA_ERR_UNSUPPORTED;

    ReorderParams p{};
    p.parents = parents;
    p.table_in = block_table;
    p.lens_in = seq_lens;
    p.spare = spare_blocks;
    p.table_out = block_table_out;
    p.lens_out = seq_lens_out;
    p.slots_out = slot_mapping_out;
    p.used_out = spare_used_out;
    p.status = dev_status;
    p.num_blocks = c.num_blocks;
    p.num_rows = num_rows;
    p.num_rows_in = num_rows_in;
    p.max_blocks = max_blocks_per_seq;
    p.block_size = c.block_size;
    p.num_kv_heads = c.num_kv_heads;
    p.row_bytes = static_cast<int32_t>(row_bytes);
    for (int first = 0; first < num_layers; first += kLayers) {
        const int n = num_layers - first < kLayers ? num_layers - first : kLayers;
        p.tables = first == 0 ? 1 : 0;
        for (int l = 0; l < n; ++l) {
            p.k[l] = caches[first + l].k_cache;
            p.v[l] = caches[first + l].v_cache;
        }
        const dim3 grid(static_cast<unsigned>(num_rows), static_cast<unsigned>(n + p.tables));
        cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        const cudaError_t e = row_bytes % 16 == 0 ? launch_pdl(beam_reorder_kernel<uint4>, grid, kThreads, 0, s, p)
                                                  : launch_pdl(beam_reorder_kernel<uint8_t>, grid, kThreads, 0, s, p);
        if (e != cudaSuccess) return PA_ERR_CUDA;
    }
    return PA_OK;
}
