// Tree decode for d_c 64, d_R 8: one CTA, cta_group::1, 128-token tiles (two
// pages), 128 MMA rows, the work list of tree_plan.cuh.
//
// A tile is 4.5 MFLOP for the tensor core (about 650 cycles in these shapes) but 16384
// exponentials (1024 cycles of the special-function units), so the softmax sets the
// pace and the kernel is built around it: two groups of four warps take alternate
// tiles, each with its own running maximum and sum and its own O accumulator (O is
// only 64 columns), so neither waits for the other until a segment ends, where the
// two meet as two partial results do. A thread reads the first 64 of its 128 scores twice from tensor
// memory, for the maximum and for the exponentials, and keeps the others. P replaces
// the scores in their own buffer, as bf16 pairs, the value product's A operand: no
// shared-memory copy of it. Three score buffers let the score products run ahead, and
// the two products are issued by a warp each, on blocking waits.
// Measured, 32 sequences of 8192 tokens, 32 heads: 135 us with 32 nodes (8 items of 128 rows a sequence,
// 111 passes over a tile per SM), 80 with 16, 64 with 12, 47 with 8 and 31 with 4 (one item, 14 passes): 1.0
// to 1.2 us a pass, about 2100 cycles, the special-function units busy half of the time and the warps
// waiting on dependent instructions the rest, and 14 us for start, switches and merge. An item costs its
// pass whatever its rows: 5 nodes (160 rows) take 45 us. One group of four warps took 162 us, one
// issuer polling for both products 146, four groups on 64-token tiles 158, two on 64-token
// tiles 184 (more waits per score), at 32 nodes. P is rounded to bf16 (half a step, 2^-8 of a weight, either
// way); the row sums add the weights as they are, in fp32.
//
// kSplit (items of at most 64 rows): query row r sits in MMA rows 32 (r / 16) + r % 16
// and the same + 16, both TMEM lanes of one warp; the first lane takes the tile's
// tokens 0..63, the second 64..127. Each writes P for its own tokens and zeros for the
// other's.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda.h>

#include "decode.cuh"

namespace mla {
namespace tsingle {
using single::D;
using single::DC;
using single::Q_LAT;
using single::Q_ROPE;
using single::ROWS;
using single::ST_LAT;
using single::ST_ROPE;
using single::STAGE_BYTES;
using single::TOK;
constexpr int THREADS = 352;                              // TMA, QK^T, 2 x 4 softmax, P.V warps
constexpr int STAGES = 8;                                 // KV ring depth
constexpr int NSB = 3;                                    // score buffers
constexpr int MIN_TILES = 2, WHOLE = 4;                   // see tree_find
// Cost of a switch, in tiles. Device times in us with 1, 3, 6, 10, 32 heads: 32 x 8192 tokens, 5 nodes: 46.0,
// 44.9, 44.4, 45.2; the same ragged: 28.9, 26.7, 24.7, 25.1; 64 ragged to 1000, 3 nodes: 20.8, 18.3, 19.4, 20.6;
// 200 ragged to 600, 8 nodes: 41.2, 36.1, 34.2, 33.8.
constexpr int GAP = 3;
constexpr uint32_t OFF_Q = 0;
constexpr uint32_t OFF_STAGE = 20480;
constexpr uint32_t OFF_MISC = OFF_STAGE + STAGES * STAGE_BYTES;
constexpr uint32_t MISC_BYTES = 5120;
constexpr uint32_t SMEM_BYTES = OFF_MISC + MISC_BYTES + 1024;   // + alignment slack
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TMEM_O = 0;                            // 64 columns per group
constexpr uint32_t TMEM_S = 128;                          // three 128-column buffers: scores, then P in the first 64
static_assert(TMEM_S + NSB * TOK <= TMEM_COLS && (OFF_STAGE % 1024) == 0 && (OFF_MISC % 1024) == 0, "layout");

struct Misc {
    uint64_t kv_full[STAGES], kv_empty[STAGES], s_full[NSB], s_free[NSB];
    uint64_t p_ready[2], pv_done[2];      // by group
    uint64_t q_ready, o_free, seg_done, drain;
    uint32_t tmem_base;
    int32_t abort_flag;
    float seg_m[2][2][ROWS], seg_l[2][2][ROWS];   // by segment parity, group and TMEM lane
    TreeWalker first;                     // the walker at its first segment
};
static_assert(sizeof(Misc) <= MISC_BYTES && SMEM_BYTES <= 232448, "misc");
}  // namespace tsingle

template <bool kSplit>
__global__ void __launch_bounds__(tsingle::THREADS, 1)
    tree_single_kernel(const __grid_constant__ CUtensorMap map_ckv, const __grid_constant__ CUtensorMap map_kr,
                       const TreeArgs args) {
    using namespace tsingle;
    constexpr int ITEM_ROWS = kSplit ? ROWS / 2 : ROWS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw_base);
    tsingle::Misc *misc = reinterpret_cast<tsingle::Misc *>(smem + OFF_MISC);
    volatile int32_t *abort_flag = &misc->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto bar = [&](const uint64_t *b) { return ptx::smem_u32(b); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            ptx::mbar_init(bar(&misc->kv_full[i]), 1);
            ptx::mbar_init(bar(&misc->kv_empty[i]), 1);
        }
        for (int i = 0; i < NSB; ++i) {
            ptx::mbar_init(bar(&misc->s_full[i]), 1);
            ptx::mbar_init(bar(&misc->s_free[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(&misc->p_ready[i]), 4);
            ptx::mbar_init(bar(&misc->pv_done[i]), 1);
        }
        ptx::mbar_init(bar(&misc->q_ready), 8);
        ptx::mbar_init(bar(&misc->o_free), 8);
        ptx::mbar_init(bar(&misc->seg_done), 8);
        ptx::mbar_init(bar(&misc->drain), 2);       // both issuers
        misc->abort_flag = 0;
        ptx::fence_mbar_init();
    }
    // zeros that are read but never written: the padded half of the RoPE K step
    for (uint32_t i = threadIdx.x; i < (STAGES + 1) * (Q_ROPE / 16); i += THREADS) {
        const uint32_t s = i / (Q_ROPE / 16), r = (i - s * (Q_ROPE / 16)) * 16;
        const uint32_t at = s == 0 ? OFF_Q + Q_LAT + Q_ROPE : OFF_STAGE + (s - 1) * STAGE_BYTES + ST_LAT + ST_ROPE;
        st_shared_v4(base + at + r, 0, 0, 0, 0);
    }
    ptx::fence_proxy_async_smem();
    if (warp == 1) {
        ptx::tmem_alloc<1>(bar(reinterpret_cast<uint64_t *>(&misc->tmem_base)), TMEM_COLS);
        ptx::tmem_relinquish<1>();
    }
    ptx::grid_dep_launch();
    if (warp == 0) {   // the plan reads only lengths, which the kernel ahead does not write
        TreeWalker w0 = tree_start(args.tree, static_cast<int32_t>(blockIdx.x), args.num_parts, TOK, ITEM_ROWS, MIN_TILES,
                                   WHOLE);
        w0.primed = w0.next();
        if (lane == 0) {
            misc->first = w0;
            if (w0.primed)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(
                    args.block_table + static_cast<int64_t>(w0.seg_b) * args.max_pages + 2 * w0.t_begin));
            ptx::prefetch_tensormap(&map_ckv);
            ptx::prefetch_tensormap(&map_kr);
        }
    }
    ptx::grid_dep_wait();   // other global memory from here on
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = misc->tmem_base;
    TreeWalker walk = misc->first;

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        if (ptx::elect_one()) {
            int32_t k = 0;
            bool bad_page = false;
            TreeShared shared = {0, 0, 0, 0};
            while (!*abort_flag && walk.next()) {
                shared = walk.shared();   // (only the last segment's can be one)
                const int32_t *trow = args.block_table + static_cast<int64_t>(walk.seg_b) * args.max_pages;
                const int32_t npages = (walk.L + 63) / 64;
                for (int32_t t = walk.t_begin; t < walk.t_end; ++t, ++k) {
                    const int s = k % STAGES;
                    const bool two = 2 * t + 1 < npages;
                    int32_t pg[2] = {trow[2 * t], two ? trow[2 * t + 1] : 0};
                    for (int i = 0; i < 2; ++i)
                        if (pg[i] < 0 || pg[i] >= args.num_pages) { bad_page = true; pg[i] = 0; }
                    if (k >= STAGES && !wait_bounded(bar(&misc->kv_empty[s]), ((k / STAGES) - 1) & 1, abort_flag,
                                                     args.timeout_ns))
                        break;
                    const uint32_t fb = bar(&misc->kv_full[s]);
                    const uint32_t npg = two ? 2u : 1u;
                    ptx::mbar_arrive_expect_tx(fb, npg * (64 * 128 + 64 * 16));
                    const uint32_t st = base + OFF_STAGE + s * STAGE_BYTES;
                    for (uint32_t i = 0; i < npg; ++i) {
                        ptx::tma_load_3d(st + i * (64 * 128), &map_ckv, fb, 0, 0, pg[i]);
                        ptx::tma_load_3d(st + ST_LAT + i * (64 * 16), &map_kr, fb, 0, 0, pg[i]);
                    }
                }
            }
            args.shared[blockIdx.x] = shared;
            if (bad_page) record_error(kErrDeviceBounds);
            for (int32_t kk = (k >= STAGES ? k - STAGES : 0); kk < k; ++kk)
                wait_bounded(bar(&misc->kv_full[kk % STAGES]), (kk / STAGES) & 1, abort_flag, args.timeout_ns);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------ QK^T issuer
        if (ptx::elect_one()) {
            const uint64_t q0 = ptx::smem_desc(base + OFF_Q, 16, 1024, ptx::kSwizzle128B);
            const uint64_t qr = ptx::smem_desc(base + OFF_Q + Q_LAT, Q_ROPE, 128, ptx::kSwizzleNone);
            const uint64_t k0 = ptx::smem_desc(base + OFF_STAGE, 16, 1024, ptx::kSwizzle128B);
            const uint64_t kr0 = ptx::smem_desc(base + OFF_STAGE + ST_LAT, ST_ROPE, 128, ptx::kSwizzleNone);
            int32_t k = 0, g = 0;
            bool ok = true;
            for (; ok && !*abort_flag && walk.next(); ++g) {
                ok = wait_bounded(bar(&misc->q_ready), g & 1, abort_flag, args.timeout_ns);
                for (int32_t t = walk.t_begin; ok && t < walk.t_end; ++t, ++k) {
                    const int ks = k % STAGES, sb = k % NSB;
                    ok = wait_bounded<false>(bar(&misc->kv_full[ks]), (k / STAGES) & 1, abort_flag, args.timeout_ns) &&
                         (k < NSB || wait_bounded<false>(bar(&misc->s_free[sb]), ((k / NSB) - 1) & 1, abort_flag,
                                                         args.timeout_ns));
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint32_t st = ks * (STAGE_BYTES >> 4);   // in the descriptors' 16-byte units
                    const uint32_t d = tmem + TMEM_S + TOK * sb;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        ptx::mma_bf16_ss<1>(d, q0 + 2 * kk, k0 + st + 2 * kk, single::IDESC_QK, kk ? 1u : 0u);
                    // RoPE step: 8 real channels + 8 zero channels, no swizzle
                    ptx::mma_bf16_ss<1>(d, qr, kr0 + st, single::IDESC_QK, 1u);
                    ptx::mma_commit(bar(&misc->s_full[sb]));
                }
            }
            ptx::mma_commit(bar(&misc->drain));   // every MMA issued is done before tensor memory is freed
            wait_bounded(bar(&misc->drain), 0, abort_flag, args.timeout_ns);
        }
    } else if (warp == 10) {
        // ------------------------------------------------------ P.V issuer
        if (ptx::elect_one()) {
            const uint64_t v0 = ptx::smem_desc(base + OFF_STAGE, 8192, 1024, ptx::kSwizzle128B);
            int32_t k = 0, g = 0;
            bool ok = true;
            for (; ok && !*abort_flag && walk.next(); ++g) {
                // the accumulators are free once the segment before has been read
                ok = g == 0 || wait_bounded(bar(&misc->o_free), (g - 1) & 1, abort_flag, args.timeout_ns);
                for (int32_t t = walk.t_begin; ok && t < walk.t_end; ++t, ++k) {
                    const int grp = k & 1, ks = k % STAGES, sb = k % NSB;
                    ok = wait_bounded(bar(&misc->p_ready[grp]), (k >> 1) & 1, abort_flag, args.timeout_ns);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint32_t d = tmem + TMEM_O + DC * grp, pa = tmem + TMEM_S + TOK * sb;
                    const uint64_t v = v0 + ks * (STAGE_BYTES >> 4);
                    const uint32_t keep = t - walk.t_begin < 2 ? 0u : 1u;   // this group's first tile of the segment
#pragma unroll
                    for (int kk = 0; kk < TOK / 16; ++kk)   // 16 tokens: 8 columns of P
                        ptx::mma_bf16_ts<1>(d, pa + 8 * kk, v + 128 * kk, single::IDESC_PV, kk ? 1u : keep);
                    ptx::mma_commit(bar(&misc->s_free[sb]));
                    ptx::mma_commit(bar(&misc->pv_done[grp]));
                    ptx::mma_commit(bar(&misc->kv_empty[ks]));
                }
            }
            ptx::mma_commit(bar(&misc->drain));
            wait_bounded(bar(&misc->drain), 0, abort_flag, args.timeout_ns);
        }
    } else {
        // ------------------------------------------------------ softmax groups
        constexpr int TT = kSplit ? TOK / 2 : TOK;             // tokens per thread and tile
        constexpr int CH = TT / 32;                            // 32-token chunks of them
        const int grp = (warp - 2) >> 2;                       // tiles k with k & 1 == grp
        const int q4 = warp & 3;                               // TMEM lane quadrant
        const int tl = q4 * 32 + lane;                         // TMEM lane = MMA row
        const int half = kSplit ? (lane >> 4) : 0;
        const int row = kSplit ? 16 * q4 + (lane & 15) : tl;   // query row of the item
        const uint32_t lane_base = static_cast<uint32_t>(q4 * 32) << 16;
        const int gtid = threadIdx.x - 64 - 128 * grp;         // 0..127 within the group
        auto arrive = [&](uint64_t *b) {
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(b));
        };
        auto load_q = [&](const TreeWalker &w) {   // by all eight warps, every load in flight at once
            const __nv_bfloat16 *qb = args.q + static_cast<int64_t>(w.row0) * D;
            constexpr int N = (ITEM_ROWS * (D / 8) + 255) / 256;   // 16-byte chunks per thread
            uint4 v[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int idx = static_cast<int>(threadIdx.x) - 64 + 256 * i;
                const int r = idx / (D / 8), cc = idx - r * (D / 8);
                v[i] = r < w.rows ? ld_global_nc_v4(qb + static_cast<int64_t>(r) * D + cc * 8) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int idx = static_cast<int>(threadIdx.x) - 64 + 256 * i;
                if (idx >= ITEM_ROWS * (D / 8)) break;
                const int r = idx / (D / 8), cc = idx - r * (D / 8);
#pragma unroll
                for (int dup = 0; dup < (kSplit ? 2 : 1); ++dup) {
                    const int m = kSplit ? 32 * (r >> 4) + (r & 15) + 16 * dup : r;   // MMA row
                    const uint32_t dst = cc < 8 ? base + OFF_Q + sw128(m, cc)
                                                : base + OFF_Q + Q_LAT + (m >> 3) * 128 + (m & 7) * 16;
                    st_shared_v4(dst, v[i].x, v[i].y, v[i].z, v[i].w);
                }
            }
            ptx::fence_proxy_async_smem();
            arrive(&misc->q_ready);
        };

        int32_t k = 0;
        int seg = 0;
        bool have = walk.next();
        if (have) load_q(walk);
        while (have && !*abort_flag) {
            const int32_t rows = walk.rows, slot = walk.slot, nodes = walk.nodes, L = walk.L;
            const int64_t out_row0 = walk.row0;
            const bool real_row = row < rows;
            const bool warp_real = (kSplit ? 16 * q4 : 32 * q4) < rows;   // warp holds a real row
            const int32_t ctx = L - nodes;
            const int32_t tok_id = real_row ? (walk.row0 + row) / args.heads : walk.first_tok;
            const int32_t node = tok_id - walk.first_tok;
            const uint32_t *mask = args.masks ? args.masks + static_cast<int64_t>(tok_id) * args.mask_words : nullptr;
            float m_run = -INFINITY, l_run = 0.f;
            bool ok = true;
            const int32_t k0 = k;
            for (int32_t t = walk.t_begin; t < walk.t_end; ++t, ++k) {
                if ((k & 1) != grp) continue;
                const int sb = k % NSB;
                const uint32_t sc = tmem + lane_base + TMEM_S + TOK * sb;
                const int32_t tok0 = t * TOK + TT * half;
                const bool edge = (t + 1) * TOK > ctx;   // the tile holds drafted tokens or the end
                uint32_t bits[CH];
                if (edge && warp_real) {
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        const int32_t d = tok0 + 32 * c - ctx;
                        bits[c] = !real_row ? 0u : d <= -32 ? ~0u : tree_bits(mask, args.mask_words, node, nodes, d);
                    }
                }
                if (!wait_bounded<false>(bar(&misc->s_full[sb]), (k / NSB) & 1, abort_flag, args.timeout_ns)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                // 64 of the thread's tokens, from token `from` on (a tensor-memory load takes one
                // column for the whole warp: with kSplit a lane loads both halves and keeps its own)
                auto scores = [&](int from, float (&x)[64]) {
                    uint32_t a[32], b[32];
                    ptx::tmem_ld32(sc + from, a);
                    ptx::tmem_ld32(sc + (kSplit ? TT : 32) + from, b);
                    ptx::tmem_wait_ld();
                    if constexpr (kSplit) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(half ? b[j] : a[j]);
                        ptx::tmem_ld32(sc + 32 + from, a);
                        ptx::tmem_ld32(sc + TT + 32 + from, b);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) x[32 + j] = __uint_as_float(half ? b[j] : a[j]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            x[j] = __uint_as_float(a[j]);
                            x[32 + j] = __uint_as_float(b[j]);
                        }
                    }
                };
                auto unseen = [&](int from, float (&x)[64]) {   // tokens that the row does not see
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        x[j] = (bits[(from + j) >> 5] >> (j & 31)) & 1u ? x[j] : -INFINITY;
                };
                // without kSplit: tokens 0..63 first, then 64..127, which stay for their exponentials
                float x[64];
                float alpha = 1.f;
                if (warp_real) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int from = 0; from < TT; from += 64) {
                        scores(from, x);
                        if (edge) {
                            // clear what is non-finite in drafted latents (QK^T has read the stage,
                            // P.V waits for p_ready; kSplit: lanes 0..15 hold other tokens than 16..31)
                            const uint32_t lanes = kSplit ? 0xFFFFu << (16 * half) : 0xFFFFFFFFu;
#pragma unroll
                            for (int c = 0; c < 64; c += 32) {
                                const int r0 = TT * half + from + c;
                                uint32_t odd = __reduce_or_sync(lanes, odd_scores(x, c, t * TOK + r0 - ctx, nodes));
                                const uint32_t st = base + OFF_STAGE + (k % STAGES) * STAGE_BYTES;
                                for (; odd; odd &= odd - 1) {
                                    const uint32_t at = st + (r0 + __ffs(odd) - 1) * 128 + (lane & 7) * 16;
                                    const uint4 w = finite_or_zero(ld_shared_v4(at));
                                    st_shared_v4(at, w.x, w.y, w.z, w.w);
                                }
                                __syncwarp();
                            }
                            unseen(from, x);
                        }
                        float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                        for (int j = 4; j < 64; j += 2) m4[(j >> 1) & 3] = fmax3(m4[(j >> 1) & 3], x[j], x[j + 1]);
                        mx = fmaxf(mx, fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]));
                    }
                    if (kSplit) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));   // the row's two halves
                    if (mx > -INFINITY &&
                        (m_run == -INFINITY || (mx - m_run) * args.scale_log2 > kRescaleThreshold)) {
                        alpha = (m_run == -INFINITY) ? 0.f : exp2f((m_run - mx) * args.scale_log2);
                        m_run = mx;
                    }
                }
                if (__any_sync(0xffffffffu, real_row && k - k0 >= 2 && alpha != 1.f)) {
                    // rescale the group's O once its last tile's P.V is done
                    if (!wait_bounded<false>(bar(&misc->pv_done[grp]), ((k >> 1) - 1) & 1, abort_flag,
                                             args.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
#pragma unroll
                    for (int cch = 0; cch < DC / 32; ++cch) {
                        uint32_t o[32];
                        const uint32_t ta = tmem + lane_base + TMEM_O + DC * grp + 32 * cch;
                        ptx::tmem_ld32(ta, o);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                        ptx::tmem_st32(ta, o);
                    }
                    ptx::tmem_wait_st();
                }
                if (warp_real) {
                    const float mb = (m_run == -INFINITY) ? 0.f : m_run * args.scale_log2;
                    float2 sum[4] = {};
                    auto weights = [&](uint32_t (&pk)[32]) {   // P of the 64 tokens in x, and their sum
#pragma unroll
                        for (int j = 0; j < 64; j += 2) {
                            const float2 a = fma_f32x2(make_float2(x[j], x[j + 1]),
                                                       make_float2(args.scale_log2, args.scale_log2),
                                                       make_float2(-mb, -mb));
                            const float2 p = make_float2(exp2f(a.x), exp2f(a.y));
                            sum[(j >> 1) & 3] = add_f32x2(sum[(j >> 1) & 3], p);
                            pk[j >> 1] = pack_bf16x2(p.x, p.y);
                        }
                    };
                    uint32_t pk[32];
                    weights(pk);
                    if constexpr (kSplit) {   // both of the row's lanes have read; each writes both K blocks
                        uint32_t w[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) w[j] = half ? 0u : pk[j];
                        ptx::tmem_st32(sc, w);
#pragma unroll
                        for (int j = 0; j < 32; ++j) w[j] = half ? pk[j] : 0u;
                        ptx::tmem_st32(sc + 32, w);
                    } else {
                        // P of tokens 64..127 goes to columns 32..63, once tokens 32..63 are read again
                        scores(0, x);
                        if (edge) unseen(0, x);
                        ptx::tmem_st32(sc + 32, pk);
                        weights(pk);
                        ptx::tmem_st32(sc, pk);
                    }
                    ptx::tmem_wait_st();
                    const float2 s2 = add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3]));
                    l_run = fmaf(l_run, alpha, s2.x + s2.y);   // (kSplit: this half's share)
                }
                // Last tile of the sequence: the stage's c_KV rows past its end (the tail of the
                // last page, or a second page not loaded) may hold any bits; P is 0 there, but
                // 0 * NaN = NaN in the value product.
                const int32_t valid = L - t * TOK;
                if (valid < TOK) {
                    const uint32_t st = base + OFF_STAGE + (k % STAGES) * STAGE_BYTES;
                    for (int idx = gtid; idx < (TOK - valid) * 8; idx += 128)
                        st_shared_v4(st + (valid + (idx >> 3)) * 128 + (idx & 7) * 16, 0u, 0u, 0u, 0u);
                }
                // P.V of the group's last tile is done by now, nearly always. Without this wait two
                // of them could be open when a segment ends, and the wait there on the last one's
                // phase parity could take the one two before for it.
                if (k >= 2 && !wait_bounded<false>(bar(&misc->pv_done[grp]), ((k >> 1) - 1) & 1, abort_flag,
                                                   args.timeout_ns)) {
                    ok = false;
                    break;
                }
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_before();
                arrive(&misc->p_ready[grp]);
            }
            if (!ok) break;

            // the segment's end: the two groups meet
            const int par = seg & 1;
            if (kSplit) l_run += __shfl_xor_sync(0xffffffffu, l_run, 16);   // the row's sum, in both lanes
            misc->seg_m[par][grp][tl] = m_run;
            misc->seg_l[par][grp][tl] = l_run;
            arrive(&misc->seg_done);
            if (!wait_bounded<false>(bar(&misc->seg_done), par, abort_flag, args.timeout_ns)) break;
            ++seg;
            have = walk.next();
            if (have) load_q(walk);   // every QK^T of the segment is done: both groups have read its scores
            // (a segment of one tile has none for one of the groups)
            const bool any0 = k - k0 >= 2 || (k0 & 1) == 0, any1 = k - k0 >= 2 || (k0 & 1) == 1;
            if (any0 && !wait_bounded<false>(bar(&misc->pv_done[0]), (((k + 1) >> 1) - 1) & 1, abort_flag, args.timeout_ns))
                break;
            if (any1 && !wait_bounded<false>(bar(&misc->pv_done[1]), ((k >> 1) - 1) & 1, abort_flag, args.timeout_ns))
                break;
            ptx::tc_fence_after();
            if (warp_real) {
                const float ma = misc->seg_m[par][0][tl], mb = misc->seg_m[par][1][tl];
                const float m = fmaxf(ma, mb);
                const float wa = ma > -INFINITY ? exp2f((ma - m) * args.scale_log2) : 0.f;
                const float wb = mb > -INFINITY ? exp2f((mb - m) * args.scale_log2) : 0.f;
                // (a group without a weight adds its sum as it is: 0, or NaN where all scores were NaN)
                const float la = misc->seg_l[par][0][tl], lb = misc->seg_l[par][1][tl];
                const float l = (ma > -INFINITY ? wa * la : la) + (mb > -INFINITY ? wb * lb : lb);
                const float inv = l > 0.f ? 1.f / l : 0.f;
                const float fa = wa * inv, fb = wb * inv;
                uint32_t oa[32], ob[32];   // this group's 32 channels of both accumulators
                ptx::tmem_ld32(tmem + lane_base + TMEM_O + 32 * grp, oa);
                ptx::tmem_ld32(tmem + lane_base + TMEM_O + DC + 32 * grp, ob);
                ptx::tmem_wait_ld();
                float o[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    o[j] = any0 ? fa * __uint_as_float(oa[j]) : 0.f;
                    if (any1) o[j] = fmaf(fb, __uint_as_float(ob[j]), o[j]);
                    if (l != l) o[j] = l;   // a NaN score makes the row NaN
                    if (kSplit) {           // tokens 0..63 first, in both lanes
                        const float other = __shfl_xor_sync(0xffffffffu, o[j], 16);
                        o[j] = half ? other + o[j] : o[j] + other;
                    }
                }
                // with kSplit a lane writes half of the channels
                constexpr int NC = kSplit ? 16 : 32;
                if (real_row) {
                    const int64_t r = slot < 0 ? out_row0 + row : static_cast<int64_t>(slot) * ITEM_ROWS + row;
                    const int64_t at = r * DC + 32 * grp + (kSplit ? 16 * half : 0);
                    if (slot < 0) {   // the whole item: final, rounded to bf16
#pragma unroll
                        for (int j = 0; j < NC; j += 8) {
                            uint32_t h[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                h[i] = kSplit && half ? pack_bf16x2(o[16 + j % 16 + 2 * i], o[16 + j % 16 + 2 * i + 1])
                                                      : pack_bf16x2(o[j + 2 * i], o[j + 2 * i + 1]);
                            *reinterpret_cast<uint4 *>(args.o_lat + at + j) = make_uint4(h[0], h[1], h[2], h[3]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < NC; j += 4)
                            *reinterpret_cast<float4 *>(args.o_part + at + j) =
                                kSplit && half ? make_float4(o[16 + j % 16], o[17 + j % 16], o[18 + j % 16], o[19 + j % 16])
                                               : make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                    }
                    if (grp == 0 && half == 0) {
                        const float lse = l != 0.f ? m * args.scale + logf(l) : -INFINITY;
                        if (slot >= 0) args.lse_part[r] = lse;
                        else if (args.lse_out) args.lse_out[r] = lse;
                    }
                }
            }
            ptx::tc_fence_before();
            arrive(&misc->o_free);
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc<1>(tmem, TMEM_COLS);
}

}  // namespace mla
