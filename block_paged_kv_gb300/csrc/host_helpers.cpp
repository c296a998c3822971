// Host helpers of the C ABI: slot mapping, its debug check, shared-prefix group
// derivation from block tables and the masks of drafted trees.  Plain C++ on host arrays.
#include <algorithm>
#include <unordered_map>
#include <unordered_set>
#include <vector>

#include "pkv.h"

extern "C" pkv_status pkv_slot_mapping_host(const int32_t *block_tables, int32_t max_blocks_per_seq,
                                            int32_t batch, int32_t num_blocks, const int32_t *rows,
                                            const int32_t *positions, int32_t n, int32_t block_size,
                                            int32_t *slots_out)
{
    if (n < 0 || block_size <= 0 || batch < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0)
        return PKV_ERR_INVALID_ARG;
    if (n > 0 && (rows == nullptr || positions == nullptr || slots_out == nullptr ||
                  block_tables == nullptr))
        return PKV_ERR_INVALID_ARG;
    bool all_ok = true;
    for (int32_t i = 0; i < n; ++i) {
        const int32_t row = rows[i], pos = positions[i];
        int32_t slot = -1;
        if (row >= 0 && row < batch && pos >= 0) {
            const int32_t logical = pos / block_size;
            if (logical < max_blocks_per_seq) {
                const int32_t phys = block_tables[static_cast<int64_t>(row) * max_blocks_per_seq + logical];
                if (phys >= 0 && phys < num_blocks &&
                    static_cast<int64_t>(phys) * block_size + block_size <= INT32_MAX)
                    slot = phys * block_size + (pos - logical * block_size);
            }
        }
        slots_out[i] = slot;
        all_ok = all_ok && slot >= 0;
    }
    return all_ok ? PKV_OK : PKV_ERR_INVALID_ARG;
}

extern "C" pkv_status pkv_slot_mapping_check_host(const int32_t *slots, int32_t n,
                                                  int32_t num_blocks, int32_t block_size,
                                                  int32_t *first_bad)
{
    if (first_bad != nullptr) *first_bad = -1;
    if (n < 0 || num_blocks <= 0 || block_size <= 0 || (n > 0 && slots == nullptr))
        return PKV_ERR_INVALID_ARG;
    const int64_t cap = static_cast<int64_t>(num_blocks) * block_size;
    std::unordered_set<int32_t> seen;
    seen.reserve(static_cast<size_t>(n));
    for (int32_t i = 0; i < n; ++i) {
        const int32_t s = slots[i];
        if (s < 0) continue;  // skipped by the append
        if (static_cast<int64_t>(s) >= cap || !seen.insert(s).second) {
            if (first_bad != nullptr) *first_bad = i;
            return PKV_ERR_INVALID_ARG;
        }
    }
    return PKV_OK;
}

extern "C" pkv_status pkv_block_copies_check_host(const int32_t *src_blocks, const int32_t *dst_blocks,
                                                  int32_t n, int32_t src_num_blocks,
                                                  int32_t dst_num_blocks, int32_t same_pool,
                                                  int32_t *first_bad)
try {
    if (first_bad != nullptr) *first_bad = -1;
    if (n < 0 || src_num_blocks <= 0 || dst_num_blocks <= 0 ||
        (n > 0 && (src_blocks == nullptr || dst_blocks == nullptr)))
        return PKV_ERR_INVALID_ARG;
    std::unordered_set<int32_t> read, written;
    for (int32_t i = 0; i < n; ++i) {
        const int32_t s = src_blocks[i], d = dst_blocks[i];
        if (s < 0 || d < 0) continue;  // skipped by the copy
        bool bad = s >= src_num_blocks || d >= dst_num_blocks;
        if (!bad && same_pool && s == d) {
            // the copy leaves it alone, but no other pair may write it
            bad = written.count(d) != 0;
        } else if (!bad) {
            bad = !written.insert(d).second || (same_pool && (read.count(d) != 0 || written.count(s) != 0));
        }
        read.insert(s);
        if (bad) {
            if (first_bad != nullptr) *first_bad = i;
            return PKV_ERR_INVALID_ARG;
        }
    }
    return PKV_OK;
} catch (...) {
    return PKV_ERR_HOST_MEMORY;
}

extern "C" int32_t pkv_prefix_groups_host(const int32_t *block_tables, int32_t max_blocks_per_seq,
                                          const int32_t *seq_lens, int32_t batch, int32_t block_size,
                                          int32_t *group_of_row, int32_t *prefix_blocks)
{
    if (batch < 0 || max_blocks_per_seq <= 0 || block_size <= 0) return -1;
    if (batch > 0 && (block_tables == nullptr || seq_lens == nullptr || group_of_row == nullptr ||
                      prefix_blocks == nullptr))
        return -1;
    auto table = [&](int32_t r) { return block_tables + static_cast<int64_t>(r) * max_blocks_per_seq; };
    // rows bucketed by their first physical block, buckets kept in order of
    // their lowest row
    std::unordered_map<int32_t, size_t> bucket_of_block;
    std::vector<std::vector<int32_t>> buckets;
    for (int32_t r = 0; r < batch; ++r) {
        group_of_row[r] = -1;
        const int32_t first = table(r)[0];
        if (first < 0) continue;
        auto it = bucket_of_block.find(first);
        if (it == bucket_of_block.end()) {
            bucket_of_block.emplace(first, buckets.size());
            buckets.push_back({r});
        } else {
            buckets[it->second].push_back(r);
        }
    }
    int32_t ngroups = 0;
    for (const auto &rows : buckets) {
        if (rows.size() < 2) continue;
        // common run against the bucket's first row, cut to full blocks
        const int32_t *lead = table(rows[0]);
        int32_t run = max_blocks_per_seq;
        for (const int32_t r : rows) {
            const int32_t *t = table(r);
            int32_t k = 0;
            const int32_t lim = std::min(run, std::max(0, seq_lens[r]) / block_size);
            while (k < lim && t[k] == lead[k]) ++k;
            run = k;
        }
        if (run <= 0) continue;
        for (const int32_t r : rows) group_of_row[r] = ngroups;
        prefix_blocks[ngroups++] = run;
    }
    return ngroups;
}

extern "C" pkv_status pkv_tree_masks_host(const int32_t *parents, const int32_t *cu_q_lens, int32_t batch,
                                          uint64_t *tree_masks)
{
    if (batch < 0 || (batch > 0 && cu_q_lens == nullptr)) return PKV_ERR_INVALID_ARG;
    for (int32_t r = 0; r < batch; ++r) {
        const int64_t n = static_cast<int64_t>(cu_q_lens[r + 1]) - cu_q_lens[r];
        if (cu_q_lens[r] < 0 || n < 0 || n > PKV_MAX_TREE || (n > 0 && (parents == nullptr || tree_masks == nullptr)))
            return PKV_ERR_INVALID_ARG;
        for (int32_t i = 0; i < n; ++i) {
            const int32_t up = parents[cu_q_lens[r] + i];
            if (up < -1 || up >= i) return PKV_ERR_INVALID_ARG;
        }
    }
    for (int32_t r = 0; r < batch; ++r) {
        uint64_t *m = tree_masks + cu_q_lens[r];
        for (int32_t i = 0; i < cu_q_lens[r + 1] - cu_q_lens[r]; ++i) {
            const int32_t up = parents[cu_q_lens[r] + i];
            m[i] = (up >= 0 ? m[up] : 0) | (1ull << i);
        }
    }
    return PKV_OK;
}
