// Host block pool: the block manager of the paged KV cache.
//
// "Как работает paged attention? (детально)" (aivaro.ru answers/837):
//   3.2 BlockManager -- a FIFO list of free physical ids, allocation takes
//       the head and sets the reference count to 1, an empty list is an
//       out-of-memory error, freeing lowers the count and returns the block
//       to the list at 0;
//   3.3 copy-on-write -- sequences that share blocks (parallel sampling, beam
//       search) copy a shared block before writing into it;
//   4.1 allocation -- logical block = pos / block_size, a new physical block
//       when the logical one is not mapped yet, the token goes to offset
//       pos % block_size;
//   4.2 deallocation.
// vLLM paper summary (easyvpn24.com/25506.html) §2-4: per-request mapping of
//   logical to physical blocks, filled left to right; a new block when the
//   last one is full; sharing between samples of one prompt.
//
// Choices where the pages leave room: an append that cannot get all of its
// blocks changes nothing (the page's sketch raises part-way through); the
// copy-on-write block is taken before the blocks for new tokens.
//
// No exception leaves an entry: what a call allocates it allocates before it
// changes anything, and PA_ERR_OOM is all that a lack of host memory does.  (The free
// list is a ring of num_blocks ids for that: giving a block back allocates nothing.)
#include <cstdint>
#include <new>
#include <unordered_map>
#include <utility>
#include <vector>

#include "pa_kv.h"

namespace {

struct Sequence {
    std::vector<int32_t> blocks;  // logical index -> physical id, -1 once released (pa_pool_release_window)
    int64_t length = 0;           // tokens held
    int64_t released_from = 0, released_to = 0;  // every block of [from, to) is released
};

struct Pool {
    int64_t num_blocks = 0;
    int32_t block_size = 0;
    std::vector<int32_t> free_ring;       // the free list: `num_free` ids from `head` on, wrapping
    int64_t head = 0, num_free = 0;
    std::vector<int32_t> ref;
    std::vector<char> reserved;  // held by the caller (pa_pool_reserve), of no sequence
    std::unordered_map<int64_t, Sequence> seqs;

    int32_t take() {
        int32_t b = free_ring[head];
        head = head + 1 == num_blocks ? 0 : head + 1;
        --num_free;
        ref[b] = 1;
        return b;
    }
    // one reference less; the last one gives the block back
    void drop(int32_t b) {
        if (--ref[b] > 0) return;
        const int64_t at = head + num_free;
        free_ring[at < num_blocks ? at : at - num_blocks] = b;
        ++num_free;
    }
};

Pool* as_pool(void* p) { return static_cast<Pool*>(p); }

}  // namespace

extern "C" {

pa_status pa_pool_create(int64_t num_blocks, int32_t block_size, const int32_t* free_order,
                         void** pool_out) {
    if (pool_out == nullptr || num_blocks <= 0 || num_blocks > INT32_MAX || block_size <= 0)
        return PA_ERR_INVALID_ARG;
    Pool* p = new (std::nothrow) Pool();
    if (p == nullptr) return PA_ERR_OOM;
    p->num_blocks = num_blocks;
    p->block_size = block_size;
    p->num_free = num_blocks;
    std::vector<char> seen;
    try {
        p->ref.assign(static_cast<size_t>(num_blocks), 0);
        p->reserved.assign(static_cast<size_t>(num_blocks), 0);
        p->free_ring.resize(static_cast<size_t>(num_blocks));
        if (free_order != nullptr) seen.assign(static_cast<size_t>(num_blocks), 0);
    } catch (const std::bad_alloc&) {
        delete p;
        return PA_ERR_OOM;
    }
    for (int64_t i = 0; i < num_blocks; ++i) {
        const int32_t b = free_order != nullptr ? free_order[i] : static_cast<int32_t>(i);
        if (free_order != nullptr) {
            if (b < 0 || b >= num_blocks || seen[b]) {
                delete p;
                return PA_ERR_INVALID_ARG;  // not a permutation
            }
            seen[b] = 1;
        }
        p->free_ring[i] = b;
    }
    *pool_out = p;
    return PA_OK;
}

void pa_pool_destroy(void* pool) { delete as_pool(pool); }

pa_status pa_pool_add_seq(void* pool, int64_t seq_id) {
    Pool* p = as_pool(pool);
    if (p == nullptr || p->seqs.count(seq_id)) return PA_ERR_INVALID_ARG;
    try {
        p->seqs.emplace(seq_id, Sequence());
    } catch (const std::bad_alloc&) {
        return PA_ERR_OOM;
    }
    return PA_OK;
}

pa_status pa_pool_append(void* pool, int64_t seq_id, int32_t n_tokens, int64_t* slots_out,
                         int32_t* cow_pairs_out, int32_t* n_cow_out) {
    Pool* p = as_pool(pool);
    if (p == nullptr || n_tokens < 0 || (n_tokens > 0 && slots_out == nullptr))
        return PA_ERR_INVALID_ARG;
    auto it = p->seqs.find(seq_id);
    if (it == p->seqs.end()) return PA_ERR_INVALID_ARG;
    Sequence& s = it->second;
    const int64_t bs = p->block_size;
    if (n_cow_out) *n_cow_out = 0;
    if (n_tokens == 0) return PA_OK;

    // blocks needed: new logical blocks, plus a private copy of a shared,
    // partially filled last block that the first new token writes into
    const int64_t blocks_after = (s.length + n_tokens + bs - 1) / bs;
    const int64_t new_blocks = blocks_after - static_cast<int64_t>(s.blocks.size());
    const bool cow = (s.length % bs) != 0 && p->ref[s.blocks.back()] > 1;
    if (new_blocks + (cow ? 1 : 0) > p->num_free) return PA_ERR_OOM;
    if (cow && (cow_pairs_out == nullptr || n_cow_out == nullptr)) return PA_ERR_INVALID_ARG;
    try {
        // (doubling, as appends of a token at a time need)
        const size_t need = static_cast<size_t>(blocks_after);
        if (need > s.blocks.capacity()) s.blocks.reserve(need > 2 * s.blocks.capacity() ? need : 2 * s.blocks.capacity());
    } catch (const std::bad_alloc&) {
        return PA_ERR_OOM;
    }

    if (cow) {
        int32_t old_b = s.blocks.back();
        int32_t new_b = p->take();
        p->ref[old_b] -= 1;
        s.blocks.back() = new_b;
        cow_pairs_out[0] = old_b;
        cow_pairs_out[1] = new_b;
        *n_cow_out = 1;
    }
    for (int32_t i = 0; i < n_tokens; ++i) {
        const int64_t pos = s.length;
        const int64_t logical = pos / bs;
        if (logical == static_cast<int64_t>(s.blocks.size())) s.blocks.push_back(p->take());
        slots_out[i] = static_cast<int64_t>(s.blocks[logical]) * bs + pos % bs;
        s.length = pos + 1;
    }
    return PA_OK;
}

pa_status pa_pool_fork(void* pool, int64_t parent, int64_t child) {
    Pool* p = as_pool(pool);
    if (p == nullptr || p->seqs.count(child)) return PA_ERR_INVALID_ARG;
    auto it = p->seqs.find(parent);
    if (it == p->seqs.end()) return PA_ERR_INVALID_ARG;
    const Sequence* held;
    try {
        Sequence copy = it->second;
        held = &p->seqs.emplace(child, std::move(copy)).first->second;
    } catch (const std::bad_alloc&) {
        return PA_ERR_OOM;
    }
    for (int32_t b : held->blocks)
        if (b >= 0) p->ref[b] += 1;
    return PA_OK;
}

pa_status pa_pool_free_seq(void* pool, int64_t seq_id) {
    Pool* p = as_pool(pool);
    if (p == nullptr) return PA_ERR_INVALID_ARG;
    auto it = p->seqs.find(seq_id);
    if (it == p->seqs.end()) return PA_ERR_INVALID_ARG;
    for (int32_t b : it->second.blocks)
        if (b >= 0) p->drop(b);
    p->seqs.erase(it);
    return PA_OK;
}

pa_status pa_pool_release_window(void* pool, int64_t seq_id, int32_t window, int32_t num_sinks,
                                 int32_t* n_released_out) {
    Pool* p = as_pool(pool);
    if (p == nullptr || window <= 0 || num_sinks < 0) return PA_ERR_INVALID_ARG;
    auto it = p->seqs.find(seq_id);
    if (it == p->seqs.end()) return PA_ERR_INVALID_ARG;
    Sequence& s = it->second;
    const int64_t bs = p->block_size;
    // blocks wholly past the sinks and wholly before what the query at position
    // length - 1 sees (later queries see no more of them); the last block stays:
    // it holds that query's own position
    const int64_t first = (static_cast<int64_t>(num_sinks) + bs - 1) / bs;
    const int64_t lo = s.length - window;
    const int64_t end = lo > 0 ? lo / bs : 0;
    int32_t n = 0;
    for (int64_t j = first; j < end; ++j) {
        // (what earlier calls released: a step looks at its new blocks alone)
        if (j >= s.released_from && j < s.released_to) j = s.released_to;
        if (j >= end) break;
        const int32_t b = s.blocks[j];
        if (b < 0) continue;
        p->drop(b);
        s.blocks[j] = -1;
        ++n;
    }
    if (first < end) {
        const bool joins = s.released_from < s.released_to && first <= s.released_to && s.released_from <= end;
        s.released_from = joins && s.released_from < first ? s.released_from : first;
        s.released_to = joins && s.released_to > end ? s.released_to : end;
    }
    if (n_released_out) *n_released_out = n;
    return PA_OK;
}

pa_status pa_pool_reserve(void* pool, int32_t n, int32_t* blocks_out) {
    Pool* p = as_pool(pool);
    if (p == nullptr || n < 0 || (n > 0 && blocks_out == nullptr)) return PA_ERR_INVALID_ARG;
    if (n > p->num_free) return PA_ERR_OOM;
    for (int32_t i = 0; i < n; ++i) {
        blocks_out[i] = p->take();
        p->reserved[blocks_out[i]] = 1;
    }
    return PA_OK;
}

pa_status pa_pool_unreserve(void* pool, const int32_t* blocks, int32_t n) {
    Pool* p = as_pool(pool);
    if (p == nullptr || n < 0 || (n > 0 && blocks == nullptr)) return PA_ERR_INVALID_ARG;
    // every id a reserved block's, and once (2: met)
    int32_t met = 0;
    while (met < n && blocks[met] >= 0 && blocks[met] < p->num_blocks && p->reserved[blocks[met]] == 1)
        p->reserved[blocks[met++]] = 2;
    for (int32_t i = 0; i < met; ++i) p->reserved[blocks[i]] = 1;
    if (met < n) return PA_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n; ++i) {
        p->reserved[blocks[i]] = 0;
        p->drop(blocks[i]);
    }
    return PA_OK;
}

// The host's half of pa_beam_reorder, by the same rule (row i and its parent's first
// child), so both sides come to the same tables without exchanging them.  Everything is
// checked and allocated before anything changes.
pa_status pa_pool_reorder(void* pool, const int64_t* old_ids, int32_t num_old, const int64_t* new_ids, int32_t num_new,
                          const int32_t* parents, const int32_t* spare_blocks, int64_t* slots_out,
                          int32_t* spare_used_out) {
    Pool* p = as_pool(pool);
    if (p == nullptr || num_old < 0 || num_new < 0 || (num_old > 0 && old_ids == nullptr) ||
        (num_new > 0 && (new_ids == nullptr || parents == nullptr || spare_blocks == nullptr)))
        return PA_ERR_INVALID_ARG;
    const int64_t bs = p->block_size;
    std::vector<int64_t> added;  // new ids entered so far
    try {
        std::unordered_map<int64_t, int> old_at, new_at;
        std::vector<Sequence*> old_seqs(static_cast<size_t>(num_old));
        for (int32_t i = 0; i < num_old; ++i) {
            auto it = p->seqs.find(old_ids[i]);
            if (it == p->seqs.end() || !old_at.emplace(old_ids[i], i).second) return PA_ERR_INVALID_ARG;
            old_seqs[i] = &it->second;
        }
        std::vector<Sequence> next(static_cast<size_t>(num_new));
        std::vector<char> fresh(static_cast<size_t>(num_new), 0), kept(static_cast<size_t>(num_old), 0);
        std::unordered_map<int32_t, int> spares;
        for (int32_t i = 0; i < num_new; ++i) {
            const bool known = p->seqs.count(new_ids[i]) != 0;
            if (!new_at.emplace(new_ids[i], i).second || (known && !old_at.count(new_ids[i])) || parents[i] >= num_old)
                return PA_ERR_INVALID_ARG;
            if (parents[i] < 0) continue;
            const Sequence& from = *old_seqs[parents[i]];
            const int64_t rest = from.length % bs;
            // a partly filled block that another sequence holds too is not the beam's
            // to write into
            if (from.length >= INT32_MAX || (rest != 0 && p->ref[from.blocks.back()] != 1)) return PA_ERR_INVALID_ARG;
            fresh[i] = rest == 0 || kept[parents[i]];
            kept[parents[i]] = 1;
            if (fresh[i] && (spare_blocks[i] < 0 || spare_blocks[i] >= p->num_blocks ||
                             p->reserved[spare_blocks[i]] != 1 || !spares.emplace(spare_blocks[i], i).second))
                return PA_ERR_INVALID_ARG;
            next[i].blocks.reserve(from.blocks.size() + (rest == 0));
            next[i] = from;
            if (rest == 0) next[i].blocks.push_back(spare_blocks[i]);
            else if (fresh[i]) next[i].blocks.back() = spare_blocks[i];
            ++next[i].length;
        }
        added.reserve(static_cast<size_t>(num_new));
        for (int32_t i = 0; i < num_new; ++i)
            if (p->seqs.emplace(new_ids[i], Sequence()).second) added.push_back(new_ids[i]);
        // ---- nothing below fails ----
        for (int32_t i = 0; i < num_new; ++i) {
            const Sequence& s = next[i];
            for (int32_t b : s.blocks)
                if (b >= 0) p->ref[b] += 1;
            if (fresh[i]) {
                p->reserved[spare_blocks[i]] = 0;
                p->ref[spare_blocks[i]] = 1;
            }
            if (slots_out != nullptr)
                slots_out[i] = parents[i] < 0 ? -1 : static_cast<int64_t>(s.blocks.back()) * bs + (s.length - 1) % bs;
            if (spare_used_out != nullptr) spare_used_out[i] = fresh[i];
        }
        for (int32_t i = 0; i < num_old; ++i) {
            for (int32_t b : old_seqs[i]->blocks)
                if (b >= 0) p->drop(b);
            if (new_at.count(old_ids[i]) == 0) p->seqs.erase(old_ids[i]);
        }
        for (int32_t i = 0; i < num_new; ++i) p->seqs.find(new_ids[i])->second = std::move(next[i]);
    } catch (const std::bad_alloc&) {
        for (int64_t id : added) p->seqs.erase(id);
        return PA_ERR_OOM;
    }
    return PA_OK;
}

pa_status pa_pool_block_table(void* pool, const int64_t* seq_ids, int32_t n, int32_t max_blocks,
                              int32_t* table_out, int32_t* lens_out) {
    Pool* p = as_pool(pool);
    if (p == nullptr || n < 0 || max_blocks < 0 || (n > 0 && (seq_ids == nullptr || table_out == nullptr)))
        return PA_ERR_INVALID_ARG;
    for (int32_t r = 0; r < n; ++r) {
        auto it = p->seqs.find(seq_ids[r]);
        if (it == p->seqs.end()) return PA_ERR_INVALID_ARG;
        const Sequence& s = it->second;
        if (static_cast<int64_t>(s.blocks.size()) > max_blocks) return PA_ERR_INVALID_ARG;
        int32_t* row = table_out + static_cast<int64_t>(r) * max_blocks;
        for (int32_t j = 0; j < max_blocks; ++j)
            row[j] = j < static_cast<int32_t>(s.blocks.size()) ? s.blocks[j] : -1;
        if (lens_out) lens_out[r] = static_cast<int32_t>(s.length);
    }
    return PA_OK;
}

int64_t pa_pool_num_free(void* pool) {
    Pool* p = as_pool(pool);
    return p ? p->num_free : -1;
}

int32_t pa_pool_ref_count(void* pool, int64_t block) {
    Pool* p = as_pool(pool);
    if (p == nullptr || block < 0 || block >= p->num_blocks) return -1;
    return p->ref[block];
}

pa_status pa_slot_mapping(const int32_t* block_table, int32_t num_seqs, int32_t max_blocks,
                          int32_t block_size, const int32_t* seq_idx, const int64_t* pos, int64_t n,
                          int64_t* slots_out) {
    if (n < 0 || num_seqs < 0 || max_blocks < 0 || block_size <= 0 ||
        (n > 0 && (block_table == nullptr || seq_idx == nullptr || pos == nullptr || slots_out == nullptr)))
        return PA_ERR_INVALID_ARG;
    for (int64_t i = 0; i < n; ++i) {
        const int32_t b = seq_idx[i];
        if (b < 0 || b >= num_seqs || pos[i] < 0) return PA_ERR_INVALID_ARG;
        const int64_t logical = pos[i] / block_size;
        const int32_t phys = logical < max_blocks
                                 ? block_table[static_cast<int64_t>(b) * max_blocks + logical]
                                 : -1;
        slots_out[i] = phys < 0 ? -1 : static_cast<int64_t>(phys) * block_size + pos[i] % block_size;
    }
    return PA_OK;
}

int32_t pa_pool_seq_len(void* pool, int64_t seq_id) {
    Pool* p = as_pool(pool);
    if (p == nullptr) return -1;
    auto it = p->seqs.find(seq_id);
    return it == p->seqs.end() ? -1 : static_cast<int32_t>(it->second.length);
}

}  // extern "C"
