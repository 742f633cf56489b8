// Host side of include/mla_step.h. Included by mla_api.cu, whose helpers it uses.
#pragma once
#include "mla_step.h"
#include "step_kernels.cuh"
#include "tree_combine.cuh"
#include "tree_single.cuh"

namespace {

// Dynamic shared memory of the step kernels, set once per device.
struct StepDeviceState {
    std::once_flag once;
    mla_status status = MLA_OK;
};
StepDeviceState g_step_dev[kMaxDevices];

mla_status step_ready() {
    mla_status st = device_ready();
    if (st != MLA_OK) return st;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MLA_ERR_CUDA;
    StepDeviceState &s = g_step_dev[dev];
    std::call_once(s.once, [&] {
        auto big = [&](const void *k, uint32_t bytes) {
            return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
        };
        auto carve = [&](const void *k) {   // as the decode step's other kernels
            return cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout,
                                        cudaSharedmemCarveoutMaxShared) == cudaSuccess;
        };
        const void *pair = reinterpret_cast<const void *>(mla::decode_pair_kernel<false, true>);
        const void *pair8 = reinterpret_cast<const void *>(mla::decode_pair_kernel<true, true>);
        const void *one = reinterpret_cast<const void *>(mla::tree_single_kernel<false>);
        const void *split = reinterpret_cast<const void *>(mla::tree_single_kernel<true>);
        const void *merge = reinterpret_cast<const void *>(mla::tree_combine_kernel);
        const void *plan = reinterpret_cast<const void *>(mla::step_plan_kernel);
        if (!big(pair, mla::pair::SMEM_BYTES) || !big(pair8, mla::pair::SMEM_BYTES) ||
            !big(one, mla::tsingle::SMEM_BYTES) || !big(split, mla::tsingle::SMEM_BYTES) ||
            !big(plan, mla::plan_smem_bytes(mla::kPlanMaxBatch)) || !carve(pair) || !carve(pair8) || !carve(one) ||
            !carve(split) || !carve(merge))
            s.status = MLA_ERR_CUDA;
    });
    return s.status;
}

mla_status check_code_pool(const mla_pool *p, int32_t channels) {
    if (!p || !p->base || !aligned(p->base, 16) || p->token_stride < channels ||
        p->page_stride < 64 * p->token_stride || (p->token_stride % 16) || (p->page_stride % 16))
        return MLA_ERR_INVALID_ARG;
    return MLA_OK;
}

mla_status append_slots(const mla_dims *dims, const void *ckv_new, int64_t ckv_new_stride, const void *kr_new,
                        int64_t kr_new_stride, const int64_t *slots, const int32_t *positions,
                        const double *inv_freq, float mscale, int32_t layout, int32_t num_tokens,
                        const mla_pool *ckv, const mla_pool *ckv8, float *scales, const mla_pool *kr,
                        int32_t num_pages, void *stream) {
    mla_status st = check_dims(dims, false);
    if (st != MLA_OK) return st;
    if (dims->page_size != 64 || (ckv8 && dims->d_latent % 16)) return MLA_ERR_UNSUPPORTED;
    if (num_tokens < 0 || num_pages <= 0 || (layout != MLA_ROPE_INTERLEAVED && layout != MLA_ROPE_HALF))
        return MLA_ERR_INVALID_ARG;
    if (num_tokens == 0) return MLA_OK;
    if (num_tokens == 1) {   // a stride that does not matter
        ckv_new_stride = dims->d_latent;
        kr_new_stride = dims->d_rope;
    }
    if (!ckv_new || !kr_new || !slots || (positions && !inv_freq)) return MLA_ERR_INVALID_ARG;
    if (!aligned(ckv_new, 16) || (ckv_new_stride % 8) || ckv_new_stride < dims->d_latent ||
        kr_new_stride < dims->d_rope || !aligned(kr_new, 2) || !aligned(slots, 8) || !aligned(positions, 4) ||
        !aligned(inv_freq, 8) || !std::isfinite(mscale))
        return MLA_ERR_INVALID_ARG;
    if (ckv8) {
        if ((st = check_code_pool(ckv8, dims->d_latent)) != MLA_OK) return st;
        if (!scales || !aligned(scales, 4)) return MLA_ERR_INVALID_ARG;
    } else if ((st = check_pool(ckv, dims->d_latent)) != MLA_OK) {
        return st;
    }
    if ((st = check_pool(kr, dims->d_rope)) != MLA_OK) return st;
    if ((st = step_ready()) != MLA_OK) return st;
    const mla_pool *c = ckv8 ? ckv8 : ckv;
    mla::AppendSlotsArgs a;
    a.ckv_new = static_cast<const __nv_bfloat16 *>(ckv_new);
    a.kr_new = static_cast<const __nv_bfloat16 *>(kr_new);
    a.ckv_new_stride = ckv_new_stride;
    a.kr_new_stride = kr_new_stride;
    a.slots = slots;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.ckv = ckv8 ? nullptr : static_cast<__nv_bfloat16 *>(const_cast<void *>(c->base));
    a.ckv8 = ckv8 ? static_cast<uint8_t *>(const_cast<void *>(c->base)) : nullptr;
    a.scales = scales;
    a.kr = static_cast<__nv_bfloat16 *>(const_cast<void *>(kr->base));
    a.ckv_page_stride = c->page_stride;
    a.ckv_token_stride = c->token_stride;
    a.kr_page_stride = kr->page_stride;
    a.kr_token_stride = kr->token_stride;
    a.mscale = mscale;
    a.T = num_tokens;
    a.d_c = dims->d_latent;
    a.d_r = dims->d_rope;
    a.num_pages = num_pages;
    a.half_layout = layout == MLA_ROPE_HALF;
    return launch_pdl(mla::append_slots_kernel, dim3(static_cast<unsigned>((int64_t(num_tokens) + 7) / 8)), dim3(256),
                      0, static_cast<cudaStream_t>(stream), a);
}

constexpr int32_t kTreeMaxPages = (1 << 25) - 1;   // token indices, rounded up to a tile, fit 31 bits

// Both cache formats of mla_decode_tree: ckv, or ckv8 and scales.
mla_status decode_tree(const mla_dims *dims, const void *q, int32_t num_tokens, const mla_pool *ckv,
                       const mla_pool *ckv8, const float *scales, const mla_pool *kr, int32_t num_pages,
                       const int32_t *block_table, int32_t max_pages, const int32_t *seq_lens,
                       const int32_t *cu_tokens, int32_t batch, const uint32_t *masks, int32_t max_nodes,
                       int32_t num_parts, void *workspace, size_t workspace_bytes, void *o_lat, float *lse_out,
                       void *stream) {
    if (!dims) return MLA_ERR_INVALID_ARG;
    mla_dims one = *dims;
    one.n_q = 1;
    mla_status st = check_dims(&one, true);
    if (st != MLA_OK) return st;
    const bool pair = variant_of(&one) == Variant::Pair512;
    if (ckv8 && !pair) return MLA_ERR_UNSUPPORTED;
    const int32_t H = one.num_heads, dc = one.d_latent;
    if (batch < 0 || num_tokens < 0 || num_parts <= 0 || max_pages <= 0 || num_pages <= 0 || max_nodes <= 0 ||
        max_nodes > MLA_TREE_MAX_NODES)
        return MLA_ERR_INVALID_ARG;
    if (batch == 0 || num_tokens == 0) return MLA_OK;
    if (!q || !block_table || !seq_lens || !cu_tokens || !workspace || !o_lat) return MLA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_tokens, 4) ||
        !aligned(masks, 4) || !aligned(workspace, 256) || !aligned(o_lat, 16) || !aligned(lse_out, 4))
        return MLA_ERR_INVALID_ARG;
    if (ckv8) {
        if ((st = check_code_pool(ckv8, dc)) != MLA_OK) return st;
        if (!scales || !aligned(scales, 16)) return MLA_ERR_INVALID_ARG;
    } else if ((st = check_pool(ckv, dc)) != MLA_OK) {
        return st;
    }
    if ((st = check_pool(kr, one.d_rope)) != MLA_OK) return st;
    const int64_t rows = static_cast<int64_t>(num_tokens) * H;
    const double cost = (static_cast<double>(rows) / 64 + batch) * (static_cast<double>(max_pages) + 16);
    if (rows >= (int64_t(1) << 31) || cost >= 2147483648.0 || num_parts > (1 << 20) || max_pages >= kTreeMaxPages)
        return MLA_ERR_UNSUPPORTED;
    if (workspace_bytes < mla_tree_workspace_bytes(&one, num_parts)) return MLA_ERR_INVALID_ARG;
    if ((st = step_ready()) != MLA_OK) return st;

    const int64_t slots = 2 * static_cast<int64_t>(num_parts);
    mla::TreeArgs a = {};
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.kv_scales = scales;
    a.o_part = static_cast<float *>(workspace);
    a.lse_part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + slots * 128 * dc * 4);
    a.timeout_ns = kDefaultTimeoutNs;
    a.max_pages = max_pages;
    a.batch = batch;
    a.num_pages = num_pages;
    a.num_parts = num_parts;
    a.n_q = 1;
    a.heads = H;
    a.scale = scale_of(&one);
    a.scale_log2 = a.scale * 1.4426950408889634f;
    a.tree = {seq_lens, cu_tokens, batch, max_pages, H, num_tokens, max_nodes,
              !pair ? mla::tsingle::GAP : ckv8 ? mla::pair::TREE_GAP_FP8 : mla::pair::TREE_GAP};
    a.masks = masks;
    a.mask_words = (max_nodes + 31) / 32;
    a.o_lat = static_cast<__nv_bfloat16 *>(o_lat);
    a.lse_out = lse_out;
    a.shared = reinterpret_cast<mla::TreeShared *>(a.lse_part + slots * 128);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // The most items that these sizes can hold, and so the most partitions that the plan
    // can use: a small step launches no more (one request of 320 tokens: 13.8 us with a full
    // grid, 11.2 us with the partitions it can use).
    const int64_t most = static_cast<int64_t>(max_nodes) * H;   // rows of a sequence
    auto bound_items = [&](int64_t item_rows) {
        return std::min(rows / item_rows + batch, batch * ((most + item_rows - 1) / item_rows));
    };
    auto bound_parts = [&](int64_t items, int64_t tile_tokens, int64_t min_tiles) {
        const int64_t tiles = (static_cast<int64_t>(max_pages) * 64 + tile_tokens - 1) / tile_tokens;
        a.num_parts = static_cast<int32_t>(std::min<int64_t>(num_parts, std::max(items, items * tiles / min_tiles)));
    };
    int64_t items;
    mla::TreeCombineArgs c;
    c.o_part = a.o_part;
    c.lse_part = a.lse_part;
    c.shared = a.shared;
    c.o_lat = a.o_lat;
    c.lse_out = lse_out;
    c.d_c = dc;
    if (pair) {
        c.item_rows = mla::pair::TREE_ROWS;
        items = bound_items(c.item_rows);
        bound_parts(items, mla::pair::TOK, mla::pair::TREE_MIN_TILES);
        CUtensorMap m32, m64, mkr, mq;
        if ((st = pool_map(&mkr, kr, 64, num_pages, 64, mla::pair::OWN, CU_TENSOR_MAP_SWIZZLE_128B)) != MLA_OK)
            return st;
        // q as one plane of packed rows; rows past the end read as zeros
        const uint64_t D = static_cast<uint64_t>(dc + one.d_rope);
        if ((st = map_3d(&mq, q, D, static_cast<uint64_t>(rows), 1, D * 2, static_cast<uint64_t>(rows) * D * 2, 64,
                         mla::pair::ROWS_CTA, 1)) != MLA_OK)
            return st;
        if (ckv8) {
            CUtensorMap msc;
            if ((st = code_pool_map(&m32, ckv8, 512, num_pages, 128, mla::pair::OWN)) != MLA_OK) return st;
            if ((st = scale_map(&msc, scales, num_pages, 32)) != MLA_OK) return st;
            st = launch_pdl(mla::decode_pair_kernel<true, true>, dim3(2 * a.num_parts), dim3(mla::kPairThreadsFp8),
                            mla::pair::SMEM_BYTES, s, m32, m32, mkr, msc, mq, a);
        } else {
            if ((st = pool_map(&m32, ckv, 512, num_pages, 64, mla::pair::OWN, CU_TENSOR_MAP_SWIZZLE_128B)) != MLA_OK)
                return st;
            if ((st = pool_map(&m64, ckv, 512, num_pages, 64, mla::pair::TOK, CU_TENSOR_MAP_SWIZZLE_128B)) != MLA_OK)
                return st;
            st = launch_pdl(mla::decode_pair_kernel<false, true>, dim3(2 * a.num_parts), dim3(mla::kPairThreads),
                            mla::pair::SMEM_BYTES, s, m32, m64, mkr, mkr /* no scales */, mq, a);
        }
    } else {
        // at most 64 query rows a sequence: each row on two TMEM lanes, half the tile's tokens each
        const bool split = most <= 64;
        c.item_rows = split ? 64 : 128;
        items = bound_items(c.item_rows);
        bound_parts(items, mla::single::TOK, mla::tsingle::MIN_TILES);
        CUtensorMap mc, mkr;
        if ((st = pool_map(&mc, ckv, 64, num_pages, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B)) != MLA_OK) return st;
        if ((st = pool_map(&mkr, kr, 8, num_pages, 8, 64, CU_TENSOR_MAP_SWIZZLE_NONE)) != MLA_OK) return st;
        st = split ? launch_pdl(mla::tree_single_kernel<true>, dim3(a.num_parts), dim3(mla::tsingle::THREADS),
                                mla::tsingle::SMEM_BYTES, s, mc, mkr, a)
                   : launch_pdl(mla::tree_single_kernel<false>, dim3(a.num_parts), dim3(mla::tsingle::THREADS),
                                mla::tsingle::SMEM_BYTES, s, mc, mkr, a);
    }
    if (st != MLA_OK || a.num_parts == 1) return st;   // one partition shares nothing
    c.num_parts = a.num_parts;
    const int64_t units = std::min<int64_t>(a.num_parts - 1, items) * c.item_rows * (dc <= 128 ? 1 : dc / 128);
    const int64_t warps = mla::kTreeCombineThreads / 32;
    const int64_t ctas = std::min<int64_t>((units + warps - 1) / warps, 2 * static_cast<int64_t>(device_sms()));
    return launch_pdl(mla::tree_combine_kernel, dim3(static_cast<unsigned>(ctas)), dim3(mla::kTreeCombineThreads), 0, s, c);
}

template <typename T>
mla_status launch_rotary(const mla::RotaryArgs &a, bool half, bool vec, dim3 grid, dim3 block, uint32_t smem,
                         cudaStream_t s) {
    if (half)
        return vec ? launch_pdl(mla::rotary_kernel<T, true, true>, grid, block, smem, s, a)
                   : launch_pdl(mla::rotary_kernel<T, true, false>, grid, block, smem, s, a);
    return vec ? launch_pdl(mla::rotary_kernel<T, false, true>, grid, block, smem, s, a)
               : launch_pdl(mla::rotary_kernel<T, false, false>, grid, block, smem, s, a);
}

}  // namespace

extern "C" {

mla_status mla_step_plan(const int32_t *cached_lens, const int32_t *new_lens, int32_t batch,
                         const int32_t *free_pages, int32_t num_free, const int32_t *free_head,
                         int32_t *block_table, int32_t max_pages_per_seq, const int32_t *parents,
                         int32_t max_nodes, int32_t num_tokens, int32_t *seq_lens, int32_t *cu_tokens,
                         int32_t *seq_ids, int32_t *positions, int64_t *slots, uint32_t *masks,
                         int32_t *free_head_out, void *stream) {
    if (batch < 0 || num_free < 0 || num_tokens < 0 || max_pages_per_seq <= 0 || max_pages_per_seq > (1 << 25))
        return MLA_ERR_INVALID_ARG;
    if (batch > MLA_STEP_MAX_BATCH) return MLA_ERR_UNSUPPORTED;
    if (parents && (max_nodes <= 0 || max_nodes > MLA_TREE_MAX_NODES)) return MLA_ERR_INVALID_ARG;
    if (!free_head || !free_head_out || free_head == free_head_out || !cu_tokens) return MLA_ERR_INVALID_ARG;
    if (batch > 0 && (!cached_lens || !new_lens || !block_table || !seq_lens)) return MLA_ERR_INVALID_ARG;
    if (batch > 0 && (seq_lens == cached_lens || seq_lens == new_lens)) return MLA_ERR_INVALID_ARG;
    if (num_free > 0 && !free_pages) return MLA_ERR_INVALID_ARG;
    if (num_tokens > 0 && (!seq_ids || !positions || !slots || (parents && !masks))) return MLA_ERR_INVALID_ARG;
    if (!aligned(cached_lens, 4) || !aligned(new_lens, 4) || !aligned(free_pages, 4) || !aligned(free_head, 4) ||
        !aligned(block_table, 4) || !aligned(parents, 4) || !aligned(seq_lens, 4) || !aligned(cu_tokens, 4) ||
        !aligned(seq_ids, 4) || !aligned(positions, 4) || !aligned(slots, 8) || !aligned(masks, 4) ||
        !aligned(free_head_out, 4))
        return MLA_ERR_INVALID_ARG;
    mla_status st = step_ready();
    if (st != MLA_OK) return st;
    mla::StepPlanArgs a;
    a.cached_lens = cached_lens;
    a.new_lens = new_lens;
    a.free_pages = free_pages;
    a.free_head = free_head;
    a.parents = parents;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.cu_tokens = cu_tokens;
    a.seq_ids = seq_ids;
    a.positions = positions;
    a.slots = slots;
    a.masks = parents ? masks : nullptr;
    a.free_head_out = free_head_out;
    a.batch = batch;
    a.max_pages = max_pages_per_seq;
    a.num_free = num_free;
    a.num_tokens = num_tokens;
    a.max_nodes = parents ? max_nodes : 0;
    a.words = parents ? (max_nodes + 31) / 32 : 0;
    const int64_t work = std::max<int64_t>(num_tokens, static_cast<int64_t>(batch) + 1);
    const int64_t ctas = std::min<int64_t>((work + mla::kPlanThreads - 1) / mla::kPlanThreads,
                                           2 * static_cast<int64_t>(device_sms()));
    return launch_pdl(mla::step_plan_kernel, dim3(static_cast<unsigned>(std::max<int64_t>(ctas, 1))),
                      dim3(mla::kPlanThreads), mla::plan_smem_bytes(batch), static_cast<cudaStream_t>(stream), a);
}

mla_status mla_rope_frequencies(int32_t rot_dim, double theta, int32_t scaling, double factor, double original_max,
                                double beta_fast, double beta_slow, double *inv_freq, double *mscale) {
    if (rot_dim <= 0 || (rot_dim % 2) || !inv_freq || !mscale || !(theta > 1.0) || !std::isfinite(theta) ||
        !(factor >= 1.0) || !std::isfinite(factor) || scaling < MLA_ROPE_NONE || scaling > MLA_ROPE_YARN)
        return MLA_ERR_INVALID_ARG;
    if (scaling == MLA_ROPE_NTK && rot_dim <= 2) return MLA_ERR_INVALID_ARG;
    if (scaling == MLA_ROPE_YARN &&
        (!(original_max > 0) || !(beta_fast > 0) || !(beta_slow > 0) || !std::isfinite(original_max) ||
         !std::isfinite(beta_fast) || !std::isfinite(beta_slow)))
        return MLA_ERR_INVALID_ARG;
    const double d = rot_dim, pi = 3.14159265358979323846;
    double base = theta, lo = 0, hi = 0;
    if (scaling == MLA_ROPE_NTK) base = theta * std::pow(factor, d / (d - 2));
    if (scaling == MLA_ROPE_YARN) {
        auto turns = [&](double b) { return d * std::log(original_max / (b * 2 * pi)) / (2 * std::log(theta)); };
        lo = std::max(std::floor(turns(beta_fast)), 0.0);
        hi = std::min(std::ceil(turns(beta_slow)), d - 1);
    }
    for (int32_t i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / d);
        if (scaling == MLA_ROPE_LINEAR) f /= factor;
        if (scaling == MLA_ROPE_YARN) {
            const double r = std::min(std::max((i - lo) / std::max(hi - lo, 1e-3), 0.0), 1.0);
            f = f / factor * r + f * (1 - r);
        }
        inv_freq[i] = f;
    }
    *mscale = scaling == MLA_ROPE_YARN && factor > 1 ? 0.1 * std::log(factor) + 1 : 1.0;
    return MLA_OK;
}

mla_status mla_rotary(const mla_rotary_tensor *x, const mla_rotary_tensor *y, int32_t dtype, int32_t num_tokens,
                      int32_t width, int32_t offset, int32_t rot_dim, const int32_t *positions,
                      const double *inv_freq, float mscale, int32_t layout, int32_t inverse, void *stream) {
    if (!x || num_tokens < 0 || width <= 0 || width > 65536 || rot_dim < 2 || (rot_dim % 2) || rot_dim > 4096 ||
        offset < 0 || offset > width - rot_dim || dtype < MLA_BF16 || dtype > MLA_FP32 ||
        (layout != MLA_ROPE_INTERLEAVED && layout != MLA_ROPE_HALF) || !std::isfinite(mscale))
        return MLA_ERR_INVALID_ARG;
    const int32_t size = dtype == MLA_FP32 ? 4 : 2, half = rot_dim / 2, E = 16 / size;
    const mla_rotary_tensor *both[2] = {x, y};
    mla::RotaryArgs a = {};
    int64_t heads = 0;
    bool copy = false;   // some tensor needs its other channels copied
    bool vec = width % E == 0 && offset % E == 0 && (layout == MLA_ROPE_HALF ? half : rot_dim) % E == 0;
    mla_rotary_tensor kept[2];
    for (int i = 0; i < 2; ++i) {
        if (!both[i]) continue;
        // the stride of a dimension of one does not matter; an output whose rows fall together has none
        mla_rotary_tensor *t = &kept[i];
        *t = *both[i];
        if (num_tokens == 1) t->in_token = t->out_token = 0;
        else if (num_tokens > 1 && t->out_token == 0) return MLA_ERR_INVALID_ARG;
        if (t->heads == 1) t->in_head = t->out_head = 0;
        else if (t->heads > 1 && t->out_head == 0) return MLA_ERR_INVALID_ARG;
        if (t->heads < 0 || t->heads > 65536) return MLA_ERR_INVALID_ARG;
        if (num_tokens > 0 && t->heads > 0 && (!t->in || !t->out)) return MLA_ERR_INVALID_ARG;
        if (!aligned(t->in, size) || !aligned(t->out, size)) return MLA_ERR_INVALID_ARG;
        if (t->in && t->in == t->out && (t->in_token != t->out_token || t->in_head != t->out_head)) return MLA_ERR_INVALID_ARG;
        copy |= t->in != t->out;
        for (int64_t stride : {t->in_token, t->in_head, t->out_token, t->out_head}) vec &= stride % E == 0;
        vec &= aligned(t->in, 16) && aligned(t->out, 16);
        a.x[i] = {t->in, t->out, t->in_token, t->in_head, t->out_token, t->out_head};
        a.heads[i] = t->heads;
        heads += t->heads;
    }
    if (heads > 65536) return MLA_ERR_INVALID_ARG;
    if (heads * width > (1 << 24)) return MLA_ERR_UNSUPPORTED;
    if (num_tokens == 0 || heads == 0) return MLA_OK;
    if (!positions || !inv_freq || !aligned(positions, 4) || !aligned(inv_freq, 8)) return MLA_ERR_INVALID_ARG;
    mla_status st = step_ready();
    if (st != MLA_OK) return st;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.mscale = mscale;
    a.sign = inverse ? -1.f : 1.f;
    a.tokens = num_tokens;
    a.width = width;
    a.offset = offset;
    a.half = half;
    // Places of a head. (Where one tensor is turned in place and the other is not, both
    // copy: in place that rewrites the same values.)
    const int32_t e = vec ? E : 1;
    a.turned = !vec ? half : layout == MLA_ROPE_HALF ? half / e : rot_dim / e;
    a.copied = copy ? (width - rot_dim) / e : 0;
    if (layout == MLA_ROPE_HALF) a.copied = (a.copied + 1) / 2;   // two vectors a place
    const int64_t places = heads * (static_cast<int64_t>(a.turned) + a.copied);
    const int64_t across = (places + mla::kRotaryThreads - 1) / mla::kRotaryThreads;   // <= 65536
    if (across > 65535) return MLA_ERR_UNSUPPORTED;
    const dim3 block(static_cast<unsigned>(((places + across - 1) / across + 31) / 32 * 32));   // even shares
    // Tokens of a CTA: 16, while their table fits and eight CTAs per SM are left.
    int64_t tt = std::min<int64_t>(16, mla::kRotaryMaxTable / half);
    while (tt > 1 && (num_tokens + tt - 1) / tt * across < 8 * static_cast<int64_t>(device_sms())) tt /= 2;
    a.TT = static_cast<int32_t>(tt);
    const dim3 grid(static_cast<unsigned>((num_tokens + tt - 1) / tt), static_cast<unsigned>(across));
    const uint32_t smem = static_cast<uint32_t>(tt * half * sizeof(float2));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool h = layout == MLA_ROPE_HALF;
    if (dtype == MLA_BF16) return launch_rotary<__nv_bfloat16>(a, h, vec, grid, block, smem, s);
    if (dtype == MLA_FP16) return launch_rotary<__half>(a, h, vec, grid, block, smem, s);
    return launch_rotary<float>(a, h, vec, grid, block, smem, s);
}

mla_status mla_append_kv_slots(const mla_dims *dims, const void *ckv_new, int64_t ckv_new_stride, const void *kr_new,
                               int64_t kr_new_stride, const int64_t *slots, const int32_t *positions,
                               const double *inv_freq, float mscale, int32_t layout, int32_t num_tokens,
                               const mla_pool *ckv, const mla_pool *kr, int32_t num_pages, void *stream) {
    if (!ckv) return MLA_ERR_INVALID_ARG;
    return append_slots(dims, ckv_new, ckv_new_stride, kr_new, kr_new_stride, slots, positions, inv_freq, mscale,
                        layout, num_tokens, ckv, nullptr, nullptr, kr, num_pages, stream);
}

mla_status mla_append_kv_slots_fp8(const mla_dims *dims, const void *ckv_new, int64_t ckv_new_stride,
                                   const void *kr_new, int64_t kr_new_stride, const int64_t *slots,
                                   const int32_t *positions, const double *inv_freq, float mscale, int32_t layout,
                                   int32_t num_tokens, const mla_pool *ckv8, float *scales, const mla_pool *kr,
                                   int32_t num_pages, void *stream) {
    if (!ckv8) return MLA_ERR_INVALID_ARG;
    return append_slots(dims, ckv_new, ckv_new_stride, kr_new, kr_new_stride, slots, positions, inv_freq, mscale,
                        layout, num_tokens, nullptr, ckv8, scales, kr, num_pages, stream);
}

int32_t mla_tree_num_parts(const mla_dims *dims, int32_t num_sms) {
    if (!dims || num_sms <= 0) return 0;
    mla_dims one = *dims;
    one.n_q = 1;
    if (check_dims(&one, true) != MLA_OK) return 0;
    return std::max(1, variant_of(&one) == Variant::Pair512 ? num_sms / 2 : num_sms);
}

size_t mla_tree_workspace_bytes(const mla_dims *dims, int32_t num_parts) {
    if (!dims || num_parts <= 0) return 0;
    mla_dims one = *dims;
    one.n_q = 1;
    if (check_dims(&one, true) != MLA_OK) return 0;
    return static_cast<size_t>(2 * static_cast<int64_t>(num_parts) * 128 * (dims->d_latent + 1) * 4 +
                               static_cast<int64_t>(num_parts) * sizeof(mla::TreeShared));
}

mla_status mla_decode_tree(const mla_dims *dims, const void *q, int32_t num_tokens, const mla_pool *ckv,
                           const mla_pool *kr, int32_t num_pages, const int32_t *block_table,
                           int32_t max_pages_per_seq, const int32_t *seq_lens, const int32_t *cu_tokens,
                           int32_t batch, const uint32_t *masks, int32_t max_nodes, int32_t num_parts,
                           void *workspace, size_t workspace_bytes, void *o_lat, float *lse_out, void *stream) {
    return decode_tree(dims, q, num_tokens, ckv, nullptr, nullptr, kr, num_pages, block_table, max_pages_per_seq,
                       seq_lens, cu_tokens, batch, masks, max_nodes, num_parts, workspace, workspace_bytes, o_lat,
                       lse_out, stream);
}

mla_status mla_decode_tree_fp8(const mla_dims *dims, const void *q, int32_t num_tokens, const mla_pool *ckv8,
                               const float *scales, const mla_pool *kr, int32_t num_pages,
                               const int32_t *block_table, int32_t max_pages_per_seq, const int32_t *seq_lens,
                               const int32_t *cu_tokens, int32_t batch, const uint32_t *masks, int32_t max_nodes,
                               int32_t num_parts, void *workspace, size_t workspace_bytes, void *o_lat,
                               float *lse_out, void *stream) {
    if (!ckv8) return MLA_ERR_INVALID_ARG;
    return decode_tree(dims, q, num_tokens, nullptr, ckv8, scales, kr, num_pages, block_table, max_pages_per_seq,
                       seq_lens, cu_tokens, batch, masks, max_nodes, num_parts, workspace, workspace_bytes, o_lat,
                       lse_out, stream);
}

}  // extern "C"
