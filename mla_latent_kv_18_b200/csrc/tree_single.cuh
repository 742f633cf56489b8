// Tree decode for d_c 64, d_R 8: one CTA, cta_group::1, tiles of one page (64
// tokens), 128 MMA rows, the work list of tree_plan.cuh.
//
// A tile is 1.2 MFLOP for the tensor core (about 370 cycles in these shapes) but 8192
// exponentials (512 cycles of the special-function units), and a softmax warp alone
// issues an instruction every 7 cycles or so. So the work is spread over four groups of four
// warps, each with its own running maximum and sum and its own O accumulator (O is
// only 64 columns): none waits for another until a segment ends, where they meet as
// partial results do. A group takes every other tile's first or second 32 tokens.
// A thread holds its 32 scores in registers, and P replaces them in their own
// buffer, as bf16 pairs, the value product's A operand: no shared-memory copy of P.
// The two products are issued by a warp each, on blocking waits.
// Measured at 32 sequences of 8192 tokens, 32 heads, 32 nodes: one softmax group of
// four warps on 128-token tiles 162 us, two groups 146 us, four groups TIME_N32.
//
// kSplit (items of at most 64 rows): query row r sits in MMA rows 32 (r / 16) + r % 16
// and the same + 16, both TMEM lanes of one warp; the first lane takes the tile's
// tokens 0..31, the second 32..63, and a group takes every fourth tile. Each lane
// writes P for its own tokens and zeros for the other's.
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
constexpr int GROUPS = 4;                                 // softmax groups of four warps
constexpr int THREADS = 32 * (3 + 4 * GROUPS);            // TMA, QK^T, softmax (2..17), P.V (18)
constexpr int TOK = 64;                                   // tokens per tile (one page)
constexpr uint32_t ST_LAT = TOK * 128, ST_ROPE = TOK * 16;
constexpr uint32_t STAGE_BYTES = ST_LAT + 2 * ST_ROPE;    // the RoPE key and its zero half
constexpr int STAGES = 12;                                // KV ring depth
constexpr int NSB = 4;                                    // score buffers
constexpr int MIN_TILES = 2;                              // fewest tiles worth a partition
constexpr uint32_t OFF_Q = 0;
constexpr uint32_t OFF_STAGE = 20480;
constexpr uint32_t OFF_MISC = OFF_STAGE + STAGES * STAGE_BYTES;
constexpr uint32_t MISC_BYTES = 9216;
constexpr uint32_t SMEM_BYTES = OFF_MISC + MISC_BYTES + 1024;   // + alignment slack
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TMEM_O = 0;                            // 64 columns per group
constexpr uint32_t TMEM_S = GROUPS * DC;                  // 64-column buffers: scores, then P in place
constexpr uint32_t IDESC_QK = ptx::idesc_bf16(128, TOK, 0, 0);
constexpr uint32_t IDESC_PV = ptx::idesc_bf16(128, DC, 0, 1);
static_assert(TMEM_S + NSB * TOK <= TMEM_COLS && (OFF_STAGE % 1024) == 0 && (STAGE_BYTES % 1024) == 0 && (OFF_MISC % 1024) == 0, "layout");

struct Misc {
    uint64_t kv_full[STAGES], kv_empty[STAGES], s_full[NSB], s_free[NSB];
    uint64_t p_ready[GROUPS], pv_done[GROUPS];
    uint64_t q_ready, o_free, seg_done, drain;
    uint32_t tmem_base;
    int32_t abort_flag;
    float seg_m[2][GROUPS][ROWS], seg_l[2][GROUPS][ROWS];   // by segment parity, group and TMEM lane
    TreeWalker first;                     // the walker at its first segment
};
static_assert(sizeof(Misc) <= MISC_BYTES && SMEM_BYTES <= 232448, "misc");
}  // namespace tsingle

template <bool kSplit>
__global__ void __launch_bounds__(tsingle::THREADS, 1)
    tree_single_kernel(const __grid_constant__ CUtensorMap map_ckv, const __grid_constant__ CUtensorMap map_kr,
                       const DecodeArgs args) {
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
        for (int i = 0; i < GROUPS; ++i) {
            ptx::mbar_init(bar(&misc->p_ready[i]), 4);
            ptx::mbar_init(bar(&misc->pv_done[i]), 1);
        }
        ptx::mbar_init(bar(&misc->q_ready), 4 * GROUPS);
        ptx::mbar_init(bar(&misc->o_free), 4 * GROUPS);
        ptx::mbar_init(bar(&misc->seg_done), 4 * GROUPS);
        ptx::mbar_init(bar(&misc->drain), 2);       // both issuers
        misc->abort_flag = 0;
        ptx::fence_mbar_init();
    }
    // zeros that are read but never written: the padded half of the RoPE K step
    for (uint32_t i = threadIdx.x; i < (Q_ROPE + STAGES * ST_ROPE) / 16; i += THREADS) {
        const uint32_t j = i * 16, k = j - Q_ROPE;   // byte of Q's half, or of the stages' halves
        const uint32_t at = j < Q_ROPE ? OFF_Q + Q_LAT + Q_ROPE + j
                                       : OFF_STAGE + k / ST_ROPE * STAGE_BYTES + ST_LAT + ST_ROPE + k % ST_ROPE;
        st_shared_v4(base + at, 0, 0, 0, 0);
    }
    ptx::fence_proxy_async_smem();
    if (warp == 1) {
        ptx::tmem_alloc<1>(bar(reinterpret_cast<uint64_t *>(&misc->tmem_base)), TMEM_COLS);
        ptx::tmem_relinquish<1>();
    }
    ptx::grid_dep_launch();
    if (warp == 0) {   // the plan reads only lengths, which the kernel ahead does not write
        TreeWalker w0 = tree_start(args.tree, static_cast<int32_t>(blockIdx.x), args.num_parts, TOK, ITEM_ROWS,
                                   MIN_TILES);
        w0.primed = w0.next();
        if (lane == 0) {
            misc->first = w0;
            if (w0.primed)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(
                    args.block_table + static_cast<int64_t>(w0.seg_b) * args.max_pages + w0.t_begin));
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
            while (!*abort_flag && walk.next()) {
                const int32_t *trow = args.block_table + static_cast<int64_t>(walk.seg_b) * args.max_pages;
                for (int32_t t = walk.t_begin; t < walk.t_end; ++t, ++k) {
                    const int s = k % STAGES;
                    int32_t page = trow[t];
                    if (page < 0 || page >= args.num_pages) { bad_page = true; page = 0; }
                    if (k >= STAGES && !wait_bounded(bar(&misc->kv_empty[s]), ((k / STAGES) - 1) & 1, abort_flag,
                                                     args.timeout_ns))
                        break;
                    const uint32_t fb = bar(&misc->kv_full[s]);
                    const uint32_t st = base + OFF_STAGE + s * STAGE_BYTES;
                    ptx::mbar_arrive_expect_tx(fb, ST_LAT + ST_ROPE);
                    ptx::tma_load_3d(st, &map_ckv, fb, 0, 0, page);
                    ptx::tma_load_3d(st + ST_LAT, &map_kr, fb, 0, 0, page);
                }
            }
            if (bad_page) record_error(kErrDeviceBounds);
            for (int32_t kk = (k >= STAGES ? k - STAGES : 0); kk < k; ++kk)
                wait_bounded(bar(&misc->kv_full[kk % STAGES]), (kk / STAGES) & 1, abort_flag, args.timeout_ns);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------ QK^T issuer
        if (ptx::elect_one()) {
            int32_t k = 0, g = 0;
            bool ok = true;
            for (; ok && !*abort_flag && walk.next(); ++g) {
                ok = wait_bounded(bar(&misc->q_ready), g & 1, abort_flag, args.timeout_ns);
                for (int32_t t = walk.t_begin; ok && t < walk.t_end; ++t, ++k) {
                    const int ks = k % STAGES, sb = k % NSB;
                    ok = wait_bounded(bar(&misc->kv_full[ks]), (k / STAGES) & 1, abort_flag, args.timeout_ns) &&
                         (k < NSB ||
                          wait_bounded(bar(&misc->s_free[sb]), ((k / NSB) - 1) & 1, abort_flag, args.timeout_ns));
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint32_t st = base + OFF_STAGE + ks * STAGE_BYTES;
                    const uint32_t d = tmem + TMEM_S + TOK * sb;
                    const uint64_t q0 = ptx::smem_desc(base + OFF_Q, 16, 1024, ptx::kSwizzle128B);
                    const uint64_t k0 = ptx::smem_desc(st, 16, 1024, ptx::kSwizzle128B);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        ptx::mma_bf16_ss<1>(d, q0 + 2 * kk, k0 + 2 * kk, IDESC_QK, kk ? 1u : 0u);
                    // RoPE step: 8 real channels + 8 zero channels, no swizzle
                    ptx::mma_bf16_ss<1>(d, ptx::smem_desc(base + OFF_Q + Q_LAT, Q_ROPE, 128, ptx::kSwizzleNone),
                                        ptx::smem_desc(st + ST_LAT, ST_ROPE, 128, ptx::kSwizzleNone), IDESC_QK, 1u);
                    ptx::mma_commit(bar(&misc->s_full[sb]));
                }
            }
            ptx::mma_commit(bar(&misc->drain));   // every MMA issued is done before tensor memory is freed
            wait_bounded(bar(&misc->drain), 0, abort_flag, args.timeout_ns);
        }
    } else if (warp == 2 + 4 * GROUPS) {
        // ------------------------------------------------------ P.V issuer
        if (ptx::elect_one()) {
            int32_t k = 0, g = 0;
            bool ok = true;
            for (; ok && !*abort_flag && walk.next(); ++g) {
                // the accumulators are free once the segment before has been read
                ok = g == 0 || wait_bounded(bar(&misc->o_free), (g - 1) & 1, abort_flag, args.timeout_ns);
                for (int32_t t = walk.t_begin; ok && t < walk.t_end; ++t, ++k) {
                    const int ks = k % STAGES, sb = k % NSB;
                    const uint64_t v0 = ptx::smem_desc(base + OFF_STAGE + ks * STAGE_BYTES, 8192, 1024, ptx::kSwizzle128B);
                    if constexpr (kSplit) {
                        const int grp = k & 3;
                        ok = wait_bounded(bar(&misc->p_ready[grp]), (k >> 2) & 1, abort_flag, args.timeout_ns);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        const uint32_t d = tmem + TMEM_O + DC * grp, pa = tmem + TMEM_S + TOK * sb;
                        const uint32_t keep = t - walk.t_begin < 4 ? 0u : 1u;   // the group's first tile of the segment
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)   // 16 tokens: 8 columns of P
                            ptx::mma_bf16_ts<1>(d, pa + 8 * kk, v0 + 128 * kk, IDESC_PV, kk ? 1u : keep);
                        ptx::mma_commit(bar(&misc->pv_done[grp]));
                    } else {
                        const uint32_t keep = t - walk.t_begin < 2 ? 0u : 1u;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {   // tokens 32 h .. 32 h + 31
                            const int grp = 2 * (k & 1) + h;
                            ok = wait_bounded(bar(&misc->p_ready[grp]), (k >> 1) & 1, abort_flag, args.timeout_ns);
                            if (!ok) break;
                            ptx::tc_fence_after();
                            const uint32_t d = tmem + TMEM_O + DC * grp, pa = tmem + TMEM_S + TOK * sb + 32 * h;
#pragma unroll
                            for (int kk = 0; kk < 2; ++kk)
                                ptx::mma_bf16_ts<1>(d, pa + 8 * kk, v0 + 256 * h + 128 * kk, IDESC_PV, kk ? 1u : keep);
                            ptx::mma_commit(bar(&misc->pv_done[grp]));
                        }
                        if (!ok) break;
                    }
                    ptx::mma_commit(bar(&misc->s_free[sb]));
                    ptx::mma_commit(bar(&misc->kv_empty[ks]));
                }
            }
            ptx::mma_commit(bar(&misc->drain));
            wait_bounded(bar(&misc->drain), 0, abort_flag, args.timeout_ns);
        }
    } else {
        // ------------------------------------------------------ softmax groups
        const int grp = (warp - 2) >> 2;
        const int q4 = warp & 3;                               // TMEM lane quadrant
        const int tl = q4 * 32 + lane;                         // TMEM lane = MMA row
        const int half = kSplit ? (lane >> 4) : (grp & 1);     // this thread's tokens 32 half .. + 31 of a tile
        const int row = kSplit ? 16 * q4 + (lane & 15) : tl;   // query row of the item
        // tile k is this group's if k % PERIOD == FIRST, and then its (k / PERIOD)-th
        constexpr int PERIOD = kSplit ? 4 : 2, SHIFT = kSplit ? 2 : 1;
        const int FIRST = kSplit ? grp : grp >> 1;
        const uint32_t lane_base = static_cast<uint32_t>(q4 * 32) << 16;
        const int gtid = (threadIdx.x - 64) & 127;             // within the group
        auto arrive = [&](uint64_t *b) {
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(b));
        };
        auto load_q = [&](const TreeWalker &w) {   // by all sixteen warps, every load in flight at once
            const __nv_bfloat16 *qb = args.q + static_cast<int64_t>(w.row0) * D;
            constexpr int NT = 128 * GROUPS;
            constexpr int N = (ITEM_ROWS * (D / 8) + NT - 1) / NT;   // 16-byte chunks per thread
            uint4 v[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int idx = static_cast<int>(threadIdx.x) - 64 + NT * i;
                const int r = idx / (D / 8), cc = idx - r * (D / 8);
                v[i] = r < w.rows ? ld_global_nc_v4(qb + static_cast<int64_t>(r) * D + cc * 8) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int idx = static_cast<int>(threadIdx.x) - 64 + NT * i;
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
            const int32_t rows = walk.rows, L = walk.L;
            const bool real_row = row < rows;
            const bool warp_real = (kSplit ? 16 * q4 : 32 * q4) < rows;   // warp holds a real row
            const int32_t ctx = L - walk.nodes;
            float m_run = -INFINITY, l_run = 0.f;
            bool ok = true;
            const int32_t k0 = k, k1 = k + walk.t_end - walk.t_begin;
            int32_t kk = k0 + ((FIRST - k0) & (PERIOD - 1));   // this group's first tile of the segment
            const bool any = kk < k1;
            for (; kk < k1; kk += PERIOD) {
                const int32_t t = walk.t_begin + kk - k0;
                const int sb = kk % NSB;
                const uint32_t sc = tmem + lane_base + TMEM_S + TOK * sb;
                const bool edge = (t + 1) * TOK > ctx;   // the tile holds drafted tokens or the end
                const int32_t d = t * TOK + 32 * half - ctx;   // drafted index of the thread's first token
                uint32_t bits = 0;
                if (edge && real_row) {
                    const int32_t tok = (walk.row0 + row) / args.heads;
                    bits = d <= -32 ? ~0u
                                    : tree_bits(args.masks ? args.masks + static_cast<int64_t>(tok) * args.mask_words
                                                           : nullptr,
                                                args.mask_words, tok - walk.first_tok, walk.nodes, d);
                }
                if (!wait_bounded<false>(bar(&misc->s_full[sb]), (kk / NSB) & 1, abort_flag, args.timeout_ns)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                float x[32];
                float alpha = 1.f;
                if (warp_real) {
                    {
                        uint32_t a[32];
                        if constexpr (kSplit) {
                            // a tensor-memory load takes one column for the whole warp: every
                            // lane loads both halves and keeps its own
                            uint32_t b[32];
                            ptx::tmem_ld32(sc, a);
                            ptx::tmem_ld32(sc + 32, b);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(half ? b[j] : a[j]);
                        } else {
                            ptx::tmem_ld32(sc + 32 * half, a);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(a[j]);
                        }
                    }
                    if (edge) {
                        // clear what is non-finite in drafted latents (QK^T has read the stage, P.V
                        // waits for p_ready; kSplit: lanes 0..15 hold other tokens than 16..31)
                        const uint32_t lanes = kSplit ? 0xFFFFu << (16 * half) : 0xFFFFFFFFu;
                        uint32_t odd = __reduce_or_sync(lanes, odd_scores(x, 0, d, walk.nodes));
                        const uint32_t st = base + OFF_STAGE + (kk % STAGES) * STAGE_BYTES;
                        for (; odd; odd &= odd - 1) {
                            const uint32_t at = st + (32 * half + __ffs(odd) - 1) * 128 + (lane & 7) * 16;
                            const uint4 w = finite_or_zero(ld_shared_v4(at));
                            st_shared_v4(at, w.x, w.y, w.z, w.w);
                        }
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 32; ++j)   // tokens that the row does not see
                            x[j] = (bits >> j) & 1u ? x[j] : -INFINITY;
                    }
                    float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                    for (int j = 4; j < 32; j += 2) m4[(j >> 1) & 3] = fmax3(m4[(j >> 1) & 3], x[j], x[j + 1]);
                    float mx = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
                    if (kSplit) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));   // the row's two lanes
                    if (mx > -INFINITY &&
                        (m_run == -INFINITY || (mx - m_run) * args.scale_log2 > kRescaleThreshold)) {
                        alpha = (m_run == -INFINITY) ? 0.f : exp2f((m_run - mx) * args.scale_log2);
                        m_run = mx;
                    }
                }
                if (__any_sync(0xffffffffu, real_row && kk - k0 >= PERIOD && alpha != 1.f)) {
                    // rescale the group's O once its last tile's P.V is done
                    if (!wait_bounded<false>(bar(&misc->pv_done[grp]), ((kk >> SHIFT) - 1) & 1, abort_flag,
                                             args.timeout_ns)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
#pragma unroll 1
                    for (int cch = 0; cch < DC / 16; ++cch) {
                        uint32_t o[16];
                        const uint32_t ta = tmem + lane_base + TMEM_O + DC * grp + 16 * cch;
                        ptx::tmem_ld16(ta, o);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                        ptx::tmem_st16(ta, o);
                    }
                    ptx::tmem_wait_st();
                }
                if (warp_real) {
                    const float mb = (m_run == -INFINITY) ? 0.f : m_run * args.scale_log2;
                    float2 sum[2] = {};
                    uint32_t pk[16];
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float2 a = fma_f32x2(make_float2(x[j], x[j + 1]),
                                                   make_float2(args.scale_log2, args.scale_log2),
                                                   make_float2(-mb, -mb));
                        const float2 p = make_float2(exp2f(a.x), exp2f(a.y));
                        sum[(j >> 1) & 1] = add_f32x2(sum[(j >> 1) & 1], p);
                        pk[j >> 1] = pack_bf16x2(p.x, p.y);
                    }
                    if constexpr (kSplit) {   // (every lane of the warp has read its scores)
                        uint32_t w[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[j] = half ? 0u : pk[j];
                        ptx::tmem_st16(sc, w);
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[j] = half ? pk[j] : 0u;
                        ptx::tmem_st16(sc + 16, w);
                    } else {
                        ptx::tmem_st16(sc + 32 * half, pk);
                    }
                    ptx::tmem_wait_st();
                    const float2 s2 = add_f32x2(sum[0], sum[1]);
                    l_run = fmaf(l_run, alpha, s2.x + s2.y);   // (kSplit: this lane's share)
                }
                if (edge) {
                    // Last tile of the sequence: the stage's c_KV rows past its end may hold any
                    // bits; P is 0 there, but 0 * NaN = NaN in the value product. (Without kSplit
                    // the group's product reads its 32 tokens alone.)
                    const int32_t hi = kSplit ? TOK : 32 * half + 32;
                    const int32_t lo = max(L - t * TOK, kSplit ? 0 : 32 * half);
                    const uint32_t st = base + OFF_STAGE + (kk % STAGES) * STAGE_BYTES;
                    for (int idx = gtid; idx < (hi - lo) * 8; idx += 128)
                        st_shared_v4(st + (lo + (idx >> 3)) * 128 + (idx & 7) * 16, 0u, 0u, 0u, 0u);
                    ptx::fence_proxy_async_smem();
                }
                // P.V of the group's last tile is done by now, nearly always. Without this wait two
                // of them could be open when a segment ends, and the wait there on the last one's
                // phase parity could take the one two before for it.
                if (kk >= PERIOD && !wait_bounded<false>(bar(&misc->pv_done[grp]), ((kk >> SHIFT) - 1) & 1, abort_flag,
                                                         args.timeout_ns)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_before();
                arrive(&misc->p_ready[grp]);
            }
            if (!ok) break;
            k = k1;

            // the segment's end: the groups meet
            const int par = seg & 1;
            if (kSplit) l_run += __shfl_xor_sync(0xffffffffu, l_run, 16);   // the row's sum, in both lanes
            misc->seg_m[par][grp][tl] = m_run;
            misc->seg_l[par][grp][tl] = any ? l_run : -1.f;                 // < 0: no tile, O not written
            arrive(&misc->seg_done);
            if (!wait_bounded<false>(bar(&misc->seg_done), par, abort_flag, args.timeout_ns)) break;
            ++seg;
            const int32_t slot = walk.slot;
            const int64_t out_row0 = walk.row0;
            have = walk.next();
            if (have) load_q(walk);   // every QK^T of the segment is done: all groups have read its scores
            for (int g = 0; g < GROUPS && ok; ++g) {   // the last P.V of every group that had a tile
                const int32_t first = kSplit ? g : g >> 1;
                const int32_t n = (k1 - 1 - first) >> SHIFT;   // index of its last tile
                if (misc->seg_l[par][g][tl] >= 0.f || misc->seg_l[par][g][tl] != misc->seg_l[par][g][tl])
                    ok = wait_bounded<false>(bar(&misc->pv_done[g]), n & 1, abort_flag, args.timeout_ns);
            }
            if (!__all_sync(0xffffffffu, ok)) break;
            ptx::tc_fence_after();
            if (warp_real) {
                float m = -INFINITY;
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) m = fmaxf(m, misc->seg_m[par][g][tl]);
                // (a group without a weight adds its sum as it is: 0, or NaN where all scores were NaN)
                float l = 0.f, f[GROUPS];
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    const float mg = misc->seg_m[par][g][tl], lg = misc->seg_l[par][g][tl];
                    const float w = mg > -INFINITY ? exp2f((mg - m) * args.scale_log2) : 0.f;
                    f[g] = lg < 0.f ? -1.f : w;
                    if (!(lg < 0.f)) l += mg > -INFINITY ? w * lg : lg;
                }
                const float inv = l > 0.f ? 1.f / l : 0.f;
                float o[16];   // this group's 16 channels of every accumulator
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = 0.f;
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    uint32_t a[16];
                    ptx::tmem_ld16(tmem + lane_base + TMEM_O + DC * g + 16 * grp, a);
                    ptx::tmem_wait_ld();
                    const float w = f[g] * inv;
                    if (f[g] >= 0.f)
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = fmaf(w, __uint_as_float(a[j]), o[j]);
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    if (kSplit) {   // tokens 0..31 of the tiles first, in both lanes
                        const float other = __shfl_xor_sync(0xffffffffu, o[j], 16);
                        o[j] = half ? other + o[j] : o[j] + other;
                    }
                    if (l != l) o[j] = l;   // a NaN score makes the row NaN
                }
                // with kSplit a lane writes half of the channels
                constexpr int NC = kSplit ? 8 : 16;
                if (real_row) {
                    const int64_t r = slot < 0 ? out_row0 + row : static_cast<int64_t>(slot) * ITEM_ROWS + row;
                    const int64_t at = r * DC + 16 * grp + (kSplit ? 8 * half : 0);
                    float y[NC];
#pragma unroll
                    for (int j = 0; j < NC; ++j) y[j] = kSplit && half ? o[(NC + j) & 15] : o[j];
                    if (slot < 0) {   // the whole item: final, rounded to bf16
#pragma unroll
                        for (int j = 0; j < NC; j += 8)
                            *reinterpret_cast<uint4 *>(args.o_lat + at + j) =
                                make_uint4(pack_bf16x2(y[j], y[j + 1]), pack_bf16x2(y[j + 2], y[j + 3]),
                                           pack_bf16x2(y[j + 4], y[j + 5]), pack_bf16x2(y[j + 6], y[j + 7]));
                    } else {
#pragma unroll
                        for (int j = 0; j < NC; j += 4)
                            *reinterpret_cast<float4 *>(args.o_part + at + j) =
                                make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
                    }
                    if (grp == 0 && (!kSplit || half == 0)) {
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
