// Merge of the items that several partitions of a tree decode share
// (tree_plan.cuh): L = log sum_s exp(lse_s), o = sum_s exp(lse_s - L) o_s.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "common.cuh"
#include "tree_plan.cuh"

namespace mla {

struct TreeCombineArgs {
    const float *o_part;        // [2 num_parts, item_rows, d_c]
    const float *lse_part;      // [2 num_parts, item_rows]
    const TreeShared *shared;   // [num_parts]
    __nv_bfloat16 *o_lat;       // [total_tokens, H, d_c]
    float *lse_out;             // [total_tokens, H] or null
    int32_t d_c, item_rows, num_parts;
};

constexpr int kTreeCombineThreads = 512;

// Every CTA reads the partitions' notes of shared items, 512 at a time, and the
// warps of the grid share out the units of all of them: min(128, d_c) channels of one
// row, four a lane, with eight slots' loads in flight. An item's parts are
// read in partition order, so the result does not depend on the launch. A grid of two CTAs
// per SM is one wave, and a step that shares nothing costs one load and a scan.
// Bound by the latency of its dependent steps (notes, lse, partials) until tens of
// items are shared.
__global__ void __launch_bounds__(kTreeCombineThreads) tree_combine_kernel(const TreeCombineArgs a) {
    __shared__ TreeShared s_item[kTreeCombineThreads];
    __shared__ int32_t s_end[kTreeCombineThreads];   // units up to and with each item
    __shared__ int32_t s_warp[kTreeCombineThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t cw = a.d_c < 128 ? a.d_c : 128;   // channels of a unit
    const int32_t chunks = a.d_c / cw;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();   // notes and partials come from the kernel before
    for (int32_t base = 0; base < a.num_parts; base += kTreeCombineThreads) {
        TreeShared it = {0, 0, 0, 0};
        if (base + tid < a.num_parts) {
            const int4 v = *reinterpret_cast<const int4 *>(a.shared + base + tid);
            it = {v.x, v.y, v.z, v.w};
        }
        if (!__syncthreads_or(it.rows)) continue;
        s_item[tid] = it;
        int32_t incl = it.rows * chunks;
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        for (int w = 0; w < warp; ++w) incl += s_warp[w];
        s_end[tid] = incl;
        __syncthreads();
        const int32_t total = s_end[kTreeCombineThreads - 1];
        for (int32_t unit = blockIdx.x * (kTreeCombineThreads / 32) + warp; unit < total;
             unit += gridDim.x * (kTreeCombineThreads / 32)) {
            int32_t lo = -1, hi = kTreeCombineThreads - 1;   // the first item whose end is past the unit
            while (hi - lo > 1) {
                const int32_t mid = (lo + hi) >> 1;
                if (s_end[mid] > unit) hi = mid;
                else lo = mid;
            }
            const TreeShared q = s_item[hi];
            const int32_t p = base + hi, cnt = q.last - p + 1;
            const int32_t local = unit - (s_end[hi] - q.rows * chunks);
            const int32_t r = local / chunks, chunk = local - r * chunks, c0 = chunk * cw + 4 * lane;
            auto slot = [&](int32_t s) { return s == 0 ? q.slot : 2 * (p + s); };
            float m = -INFINITY;
            bool nan = false;
            for (int32_t s = lane; s < cnt; s += 32) {
                const float l = a.lse_part[static_cast<int64_t>(slot(s)) * a.item_rows + r];
                nan |= l != l;
                m = fmaxf(m, l);
            }
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            nan = __any_sync(0xffffffffu, nan);   // a row that sees a NaN score is NaN whoever saw it
            float z = 0.f;
            if (m > -INFINITY)
                for (int32_t s = lane; s < cnt; s += 32)
                    z += __expf(a.lse_part[static_cast<int64_t>(slot(s)) * a.item_rows + r] - m);
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
                            w[u] = -INFINITY;
                            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (s0 + u < cnt) {
                                const int64_t row = static_cast<int64_t>(slot(s0 + u)) * a.item_rows + r;
                                w[u] = a.lse_part[row];
                                v[u] = *reinterpret_cast<const float4 *>(a.o_part + row * a.d_c + c0);
                            }
                        }
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            if (w[u] == -INFINITY) continue;   // a part in which the row sees nothing
                            const float e = __expf(w[u] - L);
                            acc.x = fmaf(e, v[u].x, acc.x);
                            acc.y = fmaf(e, v[u].y, acc.y);
                            acc.z = fmaf(e, v[u].z, acc.z);
                            acc.w = fmaf(e, v[u].w, acc.w);
                        }
                    }
                }
                const __nv_bfloat162 l2 = __floats2bfloat162_rn(acc.x, acc.y), h2 = __floats2bfloat162_rn(acc.z, acc.w);
                uint2 packed;
                packed.x = *reinterpret_cast<const uint32_t *>(&l2);
                packed.y = *reinterpret_cast<const uint32_t *>(&h2);
                *reinterpret_cast<uint2 *>(a.o_lat + (static_cast<int64_t>(q.row0) + r) * a.d_c + c0) = packed;
            }
            if (a.lse_out && lane == 0 && chunk == 0) a.lse_out[q.row0 + r] = L;
        }
        __syncthreads();   // before the next items take the shared memory
    }
}

}  // namespace mla
