// Merge of the items that several partitions of a tree decode share
// (tree_plan.cuh): L = log sum_s exp(lse_s), o = sum_s exp(lse_s - L) o_s.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "common.cuh"
#include "tree_plan.cuh"

namespace mla {

struct TreeCombineArgs {
    const float *o_part;     // [2 num_parts, item_rows, d_c]
    const float *lse_part;   // [2 num_parts, item_rows]
    TreeBatch tree;
    __nv_bfloat16 *o_lat;    // [total_tokens, H, d_c]
    float *lse_out;          // [total_tokens, H] or null
    int32_t d_c, tile_tokens, item_rows, min_tiles, num_parts;
};

constexpr int kTreeCombineWarps = 16;

// grid (num_parts - 1, item_rows * (d_c / CW) / 16), 512 threads. Column p of the grid
// merges the item that begins in partition p and goes on in p + 1, if there is
// one; a warp takes CW = min(128, d_c) channels of one row, four a lane, with
// eight slots' loads in flight. The slots of an item are read in partition order,
// so the result does not depend on the launch.
// Bound by the latency of its dependent steps (plan, lse, partials) until an
// item is shared by tens of partitions.
__global__ void __launch_bounds__(32 * kTreeCombineWarps) tree_combine_kernel(const TreeCombineArgs a) {
    __shared__ int32_t s_rows, s_row0, s_slot0, s_last, s_part;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t p = blockIdx.x;
    ptx::grid_dep_launch();
    if (warp == 0) {
        // the first item that ends after the first position of partition p + 1
        const TreePlan f = tree_find(a.tree, p + 1, a.num_parts, a.tile_tokens, a.item_rows, a.min_tiles);
        if (lane == 0) {
            s_rows = 0;
            if (p + 1 < f.P) {
                const int32_t cut = static_cast<int32_t>(part_start(p + 1, f.C, f.P));
                const int32_t mine = static_cast<int32_t>(part_start(p, f.C, f.P));
                if (f.O < cut && f.O >= mine) {
                    bool bad = false;
                    const TreeSeq q = tree_seq(a.tree, f.b, a.tile_tokens, a.item_rows, &bad);
                    s_rows = min(a.item_rows, q.nodes * a.tree.heads - f.blk * a.item_rows);
                    s_row0 = q.first_tok * a.tree.heads + f.blk * a.item_rows;
                    // its part here is this partition's first segment if the item before
                    // it, one gap earlier, ends by the partition's start
                    s_slot0 = 2 * p + ((f.O == 0 || f.O - switch_cost(a.tile_tokens) <= mine) ? 0 : 1);
                    s_last = static_cast<int32_t>(part_of_tile(f.O + q.tiles - 1, f.C, f.P));
                    s_part = p;
                }
            }
        }
    }
    ptx::grid_dep_wait();   // the partials come from the kernel before
    __syncthreads();
    const int32_t cw = a.d_c < 128 ? a.d_c : 128;   // channels of a warp
    const int32_t chunks = a.d_c / cw;
    const int32_t unit = blockIdx.y * kTreeCombineWarps + warp;
    const int32_t r = unit / chunks, c0 = (unit - r * chunks) * cw + 4 * lane;
    if (r >= s_rows) return;
    const int32_t cnt = s_last - s_part + 1;
    auto slot = [&](int32_t s) { return s == 0 ? s_slot0 : 2 * (s_part + s); };
    float m = -INFINITY;
    bool nan = false;
    for (int32_t s = lane; s < cnt; s += 32) {
        const float l = a.lse_part[slot(s) * a.item_rows + r];
        nan |= l != l;
        m = fmaxf(m, l);
    }
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    nan = __any_sync(0xffffffffu, nan);   // a row that sees a NaN score is NaN in every partition's merge
    float z = 0.f;
    if (m > -INFINITY)
        for (int32_t s = lane; s < cnt; s += 32) z += __expf(a.lse_part[slot(s) * a.item_rows + r] - m);
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    const float L = nan ? NAN : (m > -INFINITY) ? m + __logf(z) : -INFINITY;
    if (4 * lane < cw) {
        constexpr int U = 8;   // slots in flight
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (L != -INFINITY) {
            for (int32_t s0 = 0; s0 < cnt; s0 += U) {
                float w[U];
                float4 v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    w[u] = 0.f;
                    v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (s0 + u < cnt) {
                        const int64_t row = static_cast<int64_t>(slot(s0 + u)) * a.item_rows + r;
                        w[u] = a.lse_part[row];
                        v[u] = *reinterpret_cast<const float4 *>(a.o_part + row * a.d_c + c0);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (s0 + u >= cnt || w[u] == -INFINITY) continue;   // a partition where the row sees nothing
                    const float e = __expf(w[u] - L);
                    acc.x = fmaf(e, v[u].x, acc.x);
                    acc.y = fmaf(e, v[u].y, acc.y);
                    acc.z = fmaf(e, v[u].z, acc.z);
                    acc.w = fmaf(e, v[u].w, acc.w);
                }
            }
        }
        const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y), hi = __floats2bfloat162_rn(acc.z, acc.w);
        uint2 packed;
        packed.x = *reinterpret_cast<const uint32_t *>(&lo);
        packed.y = *reinterpret_cast<const uint32_t *>(&hi);
        *reinterpret_cast<uint2 *>(a.o_lat + (static_cast<int64_t>(s_row0) + r) * a.d_c + c0) = packed;
    }
    if (a.lse_out && lane == 0 && c0 < cw) a.lse_out[s_row0 + r] = L;
}

}  // namespace mla
