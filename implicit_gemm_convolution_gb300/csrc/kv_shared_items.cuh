// kv_shared_items.cuh -- how the work on shared prefixes is cut: the same arithmetic for the blocks that attend
// (kv_shared.cuh) and the ones that join their parts (kv_shared_join.cu). Whole warps.
#pragma once

#include <climits>

#include "decode_device.cuh"

namespace om {

// A group of sequences: its tokens and its prefix. Rows are its tokens times the query heads of a key head. Whatever the offsets
// hold, tokens lie in the batch and positions in the table.
struct SharedGroup {
    int t0, rows, row_blocks, len;
    int units;  // tiles of the prefix
    int64_t n;  // units of all its items, [key head][row block][unit]
};
__device__ __forceinline__ SharedGroup shared_group(const SharedProblem &p, int64_t j) {
    SharedGroup g{};
    if (j >= p.groups) return g;
    const int seqs = static_cast<int>(p.seqs), tokens = static_cast<int>(p.tokens);
    const int len = p.prefix_len[j], a = min(max(p.group_at[j], 0), seqs), b = min(max(p.group_at[j + 1], a), seqs);
    const int lo = min(max(p.cu[a], 0), tokens), hi = min(max(p.cu[b], lo), tokens);
    g.t0 = lo;
    g.rows = (hi - lo) * p.group;
    g.row_blocks = (g.rows + kSharedRows - 1) / kSharedRows;
    g.len = min(max(len, 0), static_cast<int>(p.prefix_width * p.c.page));
    g.units = (g.len + kSharedTile - 1) / kSharedTile;
    g.n = static_cast<int64_t>(static_cast<int>(p.c.heads) * g.row_blocks) * g.units;
    return g;
}

// Units of all groups, 0 where they pass 32 bits (offsets that decrease count tokens twice; others the host has bounded). mine: the
// group of the lane's number.
__device__ __forceinline__ int shared_units(const SharedProblem &p, const SharedGroup &mine) {
    int64_t total = mine.n;
#pragma unroll 1
    for (int64_t j = 32 + (threadIdx.x & 31); j < p.groups; j += 32) total += shared_group(p, j).n;
    if (p.groups > 1) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    } else {
        total = __shfl_sync(0xffffffffu, total, 0);
    }
    return total > INT_MAX - (1 << 20) ? 0 : static_cast<int>(total);
}
__device__ __forceinline__ int shared_per_block(const SharedProblem &p, int total) {
    return max((total + static_cast<int>(p.blocks) - 1) / static_cast<int>(p.blocks), kSharedMinUnits);
}

// A block's part of an item: rows row0 .. row0 + rows - 1 of a group and key head, units from .. to - 1 of all `units`.
struct SharedItem {
    int group, h, t0, row0, rows, len;
    int units, from, to;
    bool at_start;  // of the block's share
};

// The parts of a block's share one after the other, by one warp.
struct SharedItems {
    SharedGroup g;
    int u, begin, stop, before, j;

    __device__ __forceinline__ void start(const SharedProblem &p, int block) {
        const int lane = threadIdx.x & 31;
        // up to 32 groups are looked up once, a lane each
        const SharedGroup mine = shared_group(p, lane);
        const int total = shared_units(p, mine), per = shared_per_block(p, total);
        begin = u = block >= (total + per - 1) / per ? total : block * per;
        stop = min(total - u, per) + u;
        before = j = 0;
        g = SharedGroup{};
        if (u >= stop) return;
#pragma unroll 1
        for (int64_t base = 0; base < p.groups; base += 32) {
            const SharedGroup here = base == 0 ? mine : shared_group(p, base + lane);
            const int n = static_cast<int>(here.n);
            int up = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, up, o);
                if (lane >= o) up += x;
            }
            const unsigned found = __ballot_sync(0xffffffffu, u < before + up);
            if (found != 0) {
                const int at = __ffs(found) - 1;
                before += __shfl_sync(0xffffffffu, up - n, at);
                j = static_cast<int>(base) + at;
                g.t0 = __shfl_sync(0xffffffffu, here.t0, at);
                g.rows = __shfl_sync(0xffffffffu, here.rows, at);
                g.row_blocks = __shfl_sync(0xffffffffu, here.row_blocks, at);
                g.len = __shfl_sync(0xffffffffu, here.len, at);
                g.units = __shfl_sync(0xffffffffu, here.units, at);
                g.n = __shfl_sync(0xffffffffu, n, at);
                break;
            }
            before += __shfl_sync(0xffffffffu, up, 31);
        }
    }
    // The next part; false behind the last.
    __device__ __forceinline__ bool next(const SharedProblem &p, SharedItem *item) {
        if (u >= stop) return false;
        while (u >= before + static_cast<int>(g.n) && j < p.groups) {
            before += static_cast<int>(g.n);
            g = shared_group(p, ++j);
        }
        const int units = max(g.units, 1), i = (u - before) / units, first = before + i * units;
        item->group = j;
        item->h = i / max(g.row_blocks, 1);
        item->t0 = g.t0;
        item->row0 = (i - item->h * g.row_blocks) * kSharedRows;
        item->rows = min(g.rows - item->row0, kSharedRows);
        item->len = g.len;
        item->units = units;
        item->from = u - first;
        item->to = min(units, stop - first);
        item->at_start = u == begin;
        u = first + item->to;
        return true;
    }
};

}  // namespace om
