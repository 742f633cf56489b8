// The work of a decode step with any number of query tokens per sequence (a tree
// or a chain of drafted tokens), cut into partitions on the device.
//
// Query tokens are packed: sequence b owns tokens cu_tokens[b] .. cu_tokens[b + 1)
// of q, its n_b newest cache entries. Its n_b H query rows (token-major, head
// minor) are cut into blocks of `item_rows`; a block against the sequence's
// cache tiles is one item. All items lie end to end on a cost axis with `gap`
// virtual tiles between consecutive ones (the Q load and the result write of a
// switch; fewer where a tile takes longer), and partition p of P owns the positions
// [p C / P, (p + 1) C / P), as in the plan of whole sequences (common.cuh). Blocks
// of one sequence are neighbours, so the partitions that work on them at the same
// time find its cache in L2.
//
// An item that one partition covers is final: its rows go straight to the output.
// Only a partition's first and last segment can belong to an item that is shared
// with a neighbour, so a partition has two partial-result slots, 2 p for its first
// segment and 2 p + 1 for a later one, whatever the batch: the workspace does not
// grow with the number of query tokens. The partition that a shared item begins in
// leaves a note of it (TreeShared) for the merge.
#pragma once
#include <cstdint>

#include "common.cuh"

namespace mla {

struct TreeBatch {
    const int32_t *seq_lens;    // [batch], the step's own tokens included
    const int32_t *cu_tokens;   // [batch + 1]
    int32_t batch, max_pages, heads, total_tokens, max_nodes;
    int32_t gap;                // cost of a switch, in tiles
};

// What sequence b asks for; a bad one (a length outside the table, more query
// tokens than max_nodes, than the sequence has or than q holds) asks for nothing.
struct TreeSeq {
    int32_t L, nodes, first_tok, tiles, blocks;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeBatch &t, int32_t b, int32_t tile_tokens, int32_t item_rows,
                                            bool *bad) {
    TreeSeq q;
    const int32_t lo = t.cu_tokens[b], hi = t.cu_tokens[b + 1];
    q.L = clamp_len(t.seq_lens[b], t.max_pages, 0, bad);
    q.first_tok = lo;
    const int64_t n = static_cast<int64_t>(hi) - lo;
    if (lo < 0 || n < 0 || hi > t.total_tokens || n > t.max_nodes || n > q.L) {
        *bad = true;
        q.nodes = 0;
    } else {
        q.nodes = static_cast<int32_t>(n);
    }
    q.tiles = static_cast<int32_t>(tiles_of_len(q.L, tile_tokens));
    q.blocks = (q.nodes * t.heads + item_rows - 1) / item_rows;
    return q;
}

// A shared item, noted by the partition that it begins in (rows 0: none): its rows
// in the output, the slot of its part there, and the last partition that has a part,
// every later one in slot 2 p.
struct TreeShared {
    int32_t row0, rows, slot, last;
};

// Walks the items of one partition; every thread that walks it gets the same
// segments. Costs fit 32 bits (checked on the host).
struct TreeWalker {
    TreeBatch batch;
    int32_t tile_tokens, item_rows, part;
    int32_t ts, tile, te;         // this partition's range on the cost axis: start, position reached, end
    int32_t C, P;                 // total cost, partitions in use
    int32_t b, blk, O;            // the next item: sequence, row block, cost offset
    bool later;                   // a segment has been handed out
    bool primed;                  // the current segment was found ahead: next() hands it out
    // current segment
    int32_t seg_b, L, nodes, first_tok, row0, rows, t_begin, t_end, slot;   // slot < 0: the whole item
    int32_t item_end;             // cost position after the item's last tile
    int32_t rot;                  // tiles skipped at first and taken last: see tile_at

    // The t-th position of the segment (t_begin <= t < t_end) as a tile. Partitions advance a tile
    // at a time together, so position x of a partition is a clock that all of them share, and a
    // segment is rotated so that position x takes tile x mod (tiles of its sequence) where it can.
    // Row blocks of one sequence, in several partitions, then read the same tile at the same time,
    // one of them from HBM and the others from L2: 4 sequences of 65536 tokens, 32 nodes of 128
    // heads, 2244 us in order and 1900 so; 32 ragged ones of up to 32768, 1279 and 1150.
    __device__ int32_t tile_at(int32_t t) const { return t + rot < t_end ? t + rot : t + rot - (t_end - t_begin); }

    // The current segment's note, if its item begins here and goes on.
    __device__ TreeShared shared() const {
        TreeShared s = {0, 0, 0, 0};
        if (slot >= 0 && t_begin == 0)
            s = {row0, rows, slot, static_cast<int32_t>(part_of_tile(item_end - 1, C, P))};
        return s;
    }

    __device__ bool next() {
        if (primed) {
            primed = false;
            return true;
        }
        while (tile < te && b < batch.batch && O < te) {
            bool bad = false;
            const TreeSeq q = tree_seq(batch, b, tile_tokens, item_rows, &bad);
            if (blk >= q.blocks) {
                ++b;
                blk = 0;
                continue;
            }
            const int32_t at = O, i = blk;
            O += q.tiles + batch.gap;
            ++blk;
            if (at + q.tiles <= tile) continue;   // the partition starts in the gap after it
            seg_b = b;
            L = q.L;
            nodes = q.nodes;
            first_tok = q.first_tok;
            row0 = q.first_tok * batch.heads + i * item_rows;
            rows = min(item_rows, q.nodes * batch.heads - i * item_rows);
            item_end = at + q.tiles;
            t_begin = max(tile - at, 0);
            t_end = min(te - at, q.tiles);
            slot = (t_begin == 0 && t_end == q.tiles) ? -1 : 2 * part + (later ? 1 : 0);
            later = true;
            tile = at + t_end;
            // the clock's tile, and after how many positions it comes to the segment's first one
            const int32_t s = (at + t_begin - ts) % q.tiles, n = t_end - t_begin;
            const int32_t d = t_begin - s + (s > t_begin ? q.tiles : 0);
            rot = s >= t_begin && s < t_end ? s - t_begin : d < n ? n - d : 0;
            return true;
        }
        return false;
    }
};

struct TreePlan {
    int32_t C, P;           // cost of all items, partitions in use
    int32_t b, blk, O;      // the first item that ends after a position: see tree_find
};

// Warp-cooperative: the plan's totals and the first item that ends after cost
// position start(part), if part < P. All 32 lanes must call it; every lane gets the
// result. Fewer partitions than num_parts are used where there is little to do: items of
// up to `whole` tiles on average are not split (a merge costs as much as some tiles: 8
// one-item sequences of 512 tokens take 17.3 us whole and 19.9 us in halves), longer
// ones into parts of `min_tiles` at least (one item of 1024 tokens: 18.6 us in parts of 8
// tiles, 15.1 us of 4; of 4096: 21.2, 20.0, and 23.2 us of 2).
__device__ inline TreePlan tree_find(const TreeBatch &t, int32_t part, int32_t num_parts, int32_t tile_tokens,
                                     int32_t item_rows, int32_t min_tiles, int32_t whole) {
    const int lane = threadIdx.x & 31;
    const int32_t W = t.gap;
    bool bad = false;
    int32_t N = 0, items = 0;
    uint32_t tokens = 0;
    TreeSeq first = {};   // this lane's sequence of the first 32, kept for the second pass
    for (int32_t base = 0; base < t.batch; base += 32) {
        const int32_t b = base + lane;
        TreeSeq q = {};
        if (b < t.batch) q = tree_seq(t, b, tile_tokens, item_rows, &bad);
        if (base == 0) first = q;
        // Where cu_tokens turns back, sequences can overlap and hold more tokens together than
        // there are; the costs would pass the 32 bits that the host has checked. Such a step is
        // not run.
        tokens += __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(q.nodes));
        if (tokens > static_cast<uint32_t>(t.total_tokens)) {
            bad = true;
            items = 0;
            break;
        }
        N += __reduce_add_sync(0xffffffffu, q.blocks * q.tiles);
        items += __reduce_add_sync(0xffffffffu, q.blocks);
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) record_error(kErrDeviceBounds);
    TreePlan r = {0, 0, t.batch, 0, 0};
    if (items == 0) return r;
    r.C = N + W * (items - 1);
    r.P = min(num_parts, N > whole * items ? N / min_tiles : items);
    if (part >= r.P) return r;
    const int32_t ts = static_cast<int32_t>(part_start(part, r.C, r.P));
    int32_t CO = 0;
    for (int32_t base = 0; base < t.batch; base += 32) {
        const int32_t b = base + lane;
        TreeSeq q = first;
        if (base > 0) {
            q = TreeSeq{};
            if (b < t.batch) q = tree_seq(t, b, tile_tokens, item_rows, &bad);
        }
        const int32_t step = q.tiles + W;
        const int32_t w = q.blocks * step;
        int32_t incl = w;
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const int32_t Cb = CO + incl - w;
        const unsigned m = __ballot_sync(0xffffffffu, q.blocks > 0 && Cb + w - W > ts);
        if (m) {
            const int src = __ffs(m) - 1;
            int32_t blk = 0, O = Cb;
            if (lane == src && ts > Cb) {
                blk = (ts - Cb) / step;
                if (ts - Cb - blk * step >= q.tiles) ++blk;   // in the gap after that block
                O = Cb + blk * step;
            }
            r.b = __shfl_sync(0xffffffffu, b, src);
            r.blk = __shfl_sync(0xffffffffu, blk, src);
            r.O = __shfl_sync(0xffffffffu, O, src);
            return r;
        }
        CO += __shfl_sync(0xffffffffu, incl, 31);
    }
    return r;
}

// The walker of partition `part`, before its first segment (warp-cooperative).
__device__ inline TreeWalker tree_start(const TreeBatch &t, int32_t part, int32_t num_parts, int32_t tile_tokens,
                                        int32_t item_rows, int32_t min_tiles, int32_t whole) {
    const TreePlan p = tree_find(t, part, num_parts, tile_tokens, item_rows, min_tiles, whole);
    TreeWalker w = {};
    w.batch = t;
    w.tile_tokens = tile_tokens;
    w.item_rows = item_rows;
    w.part = part;
    w.C = p.C;
    w.P = p.P;
    if (part < p.P) {
        w.ts = w.tile = static_cast<int32_t>(part_start(part, p.C, p.P));
        w.te = static_cast<int32_t>(part_start(part + 1, p.C, p.P));
    }
    w.b = p.b;
    w.blk = p.blk;
    w.O = p.O;
    return w;
}

}  // namespace mla
