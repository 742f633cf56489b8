// The steps around a drafted step's attention: its plan (pages, slots, tree
// masks), rotary positions, and the cache write by slot map.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "small_kernels.cuh"

namespace mla {

// ---------------------------------------------------------------------------
// Step plan. With c_b cached and n_b new tokens of sequence b, cu the exclusive
// sums of n and f those of the fresh pages ceil((c_b + n_b) / 64) - ceil(c_b / 64):
//   table[b][ceil(c_b / 64) + k] = free_pages[head + f_b + k]
//   token t = cu_b + i:  slot = page(c_b + i) * 64 + (c_b + i) % 64
//   position = c_b + depth(i);  mask_i = bit i | mask_parent(i)
// One launch, no exchange between CTAs: every CTA scans the request lengths (two
// sums, in 64 bits so that bad lengths cannot wrap) into its shared memory and then
// takes its share of the tokens, fresh pages and sequences, finding each one's
// sequence by bisection there. A request's pages come from the table (old ones,
// which no CTA writes) or straight from the free list (fresh ones).
// Bound by latency: launch, lengths, two block scans per 512 requests, one dependent
// load per token. The bytes are 16 a token.
// ---------------------------------------------------------------------------
struct StepPlanArgs {
    const int32_t *cached_lens, *new_lens;   // [batch]
    const int32_t *free_pages;               // [num_free]
    const int32_t *free_head;                // [1]
    const int32_t *parents;                  // [num_tokens] or null
    int32_t *block_table;                    // [batch, max_pages]
    int32_t *seq_lens, *cu_tokens;           // [batch], [batch + 1]
    int32_t *seq_ids, *positions;            // [num_tokens]
    int64_t *slots;                          // [num_tokens]
    uint32_t *masks;                         // [num_tokens, words] with parents
    int32_t *free_head_out;                  // [1]
    int32_t batch, max_pages, num_free, num_tokens, max_nodes, words;
};

constexpr int kPlanThreads = 512;
constexpr int kPlanMaxBatch = 16384;     // two int32 sums per sequence in shared memory
constexpr int kPlanMaxWords = 8;         // 256 tree nodes

__host__ __device__ constexpr uint32_t plan_smem_bytes(int32_t batch) { return (batch + 1) * 8u; }

// Largest b with sums[b] <= x (sums[0] = 0 <= x < sums[n]): skips empty entries.
__device__ __forceinline__ int32_t plan_find(const int32_t *sums, int32_t n, int32_t x) {
    int32_t lo = 0, hi = n;   // sums[lo] <= x < sums[hi]
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (sums[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) step_plan_kernel(const StepPlanArgs a) {
    extern __shared__ int32_t plan_smem[];
    int32_t *cu = plan_smem, *fresh = plan_smem + a.batch + 1;   // exclusive sums, totals last
    __shared__ int64_t warp_sum[2][kPlanThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t cap = static_cast<int64_t>(a.max_pages) * 64;
    const int64_t big = 0x7FFFFFFF;
    bool bad = false;
    // The kernel after this one reads the plan before its own dependency wait
    // (the decode calls' seq_lens and tables), so this one never lets it start early.
    ptx::grid_dep_wait();

    // what sequence b adds: a length that does not fit its table row adds nothing
    auto lens = [&](int32_t b, int64_t *c, int64_t *n) {
        *c = a.cached_lens[b];
        *n = a.new_lens[b];
        if (*c < 0 || *c > cap || *n < 0 || *c + *n > cap) {
            bad = true;
            *n = 0;
            *c = *c < 0 ? 0 : *c > cap ? cap : *c;
        }
    };
    int64_t carry_t = 0, carry_f = 0;
    for (int32_t b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
        const int32_t b = b0 + tid;
        int64_t c = 0, n = 0;
        if (b < a.batch) lens(b, &c, &n);
        int64_t st = n, sf = (c + n + 63) / 64 - (c + 63) / 64;
        const int64_t mt = st, mf = sf;
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t vt = __shfl_up_sync(0xffffffffu, st, o), vf = __shfl_up_sync(0xffffffffu, sf, o);
            if (lane >= o) {
                st += vt;
                sf += vf;
            }
        }
        if (lane == 31) {
            warp_sum[0][warp] = st;
            warp_sum[1][warp] = sf;
        }
        __syncthreads();
        int64_t bt = carry_t, bf = carry_f;
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            const int64_t vt = warp_sum[0][w], vf = warp_sum[1][w];
            if (w < warp) {
                bt += vt;
                bf += vf;
            }
            carry_t += vt;
            carry_f += vf;
        }
        if (b < a.batch) {
            cu[b] = static_cast<int32_t>(min(bt + st - mt, big));
            fresh[b] = static_cast<int32_t>(min(bf + sf - mf, big));
        }
        __syncthreads();
    }
    if (tid == 0) {
        cu[a.batch] = static_cast<int32_t>(min(carry_t, big));
        fresh[a.batch] = static_cast<int32_t>(min(carry_f, big));
    }
    __syncthreads();
    const int32_t total = cu[a.batch], pages = fresh[a.batch];
    int64_t head = a.free_head[0];
    if (head < 0 || head > a.num_free) {
        bad = true;
        head = head < 0 ? 0 : a.num_free;
    }
    if (total > a.num_tokens || head + pages > a.num_free) bad = true;
    auto fresh_page = [&](int64_t k) { return head + k < a.num_free ? a.free_pages[head + k] : -1; };
    const int32_t first = blockIdx.x * kPlanThreads + tid, stride = gridDim.x * kPlanThreads;

    for (int32_t t = first; t < a.num_tokens; t += stride) {
        int32_t id = -1, pos = -1;
        int64_t slot = -1;
        uint32_t mask[kPlanMaxWords] = {};
        if (t < total) {
            id = plan_find(cu, a.batch, t);
            const int32_t i = t - cu[id];
            const int64_t c = a.cached_lens[id], at = c + i;
            const int64_t pg = at / 64 - (c + 63) / 64;
            const int32_t page = pg < 0 ? a.block_table[static_cast<int64_t>(id) * a.max_pages + at / 64]
                                        : fresh_page(fresh[id] + pg);
            if (page >= 0) slot = static_cast<int64_t>(page) * 64 + at % 64;
            else bad = true;
            int32_t depth = i;
            if (a.parents) {
                // up the tree; a parent comes before its child, so this ends. An entry
                // that does not is taken for a root.
                const int32_t *par = a.parents + cu[id];
                if (i >= a.max_nodes) bad = true;
                depth = 0;
                for (int32_t j = i;;) {
#pragma unroll
                    for (int w = 0; w < kPlanMaxWords; ++w) mask[w] |= (j >> 5) == w ? 1u << (j & 31) : 0u;
                    const int32_t up = par[j];
                    if (up >= j) bad = true;
                    if (up < 0 || up >= j) break;
                    j = up;
                    ++depth;
                }
            }
            pos = static_cast<int32_t>(c + depth);
        }
        a.seq_ids[t] = id;
        a.positions[t] = pos;
        a.slots[t] = slot;
        if (a.masks) {
#pragma unroll
            for (int w = 0; w < kPlanMaxWords; ++w)
                if (w < a.words) a.masks[static_cast<int64_t>(t) * a.words + w] = mask[w];
        }
    }
    for (int32_t k = first; k < pages; k += stride) {
        const int32_t b = plan_find(fresh, a.batch, k);
        const int64_t p0 = (static_cast<int64_t>(a.cached_lens[b]) + 63) / 64;
        a.block_table[static_cast<int64_t>(b) * a.max_pages + p0 + (k - fresh[b])] = fresh_page(k);
    }
    for (int32_t b = first; b <= a.batch; b += stride) {
        a.cu_tokens[b] = cu[b];
        if (b < a.batch) {
            int64_t c, n;
            lens(b, &c, &n);
            a.seq_lens[b] = static_cast<int32_t>(c + n);
        }
    }
    if (first == 0) a.free_head_out[0] = static_cast<int32_t>(min(head + pages, static_cast<int64_t>(a.num_free)));
    if (bad) record_error(kErrDeviceBounds);
    __threadfence();   // the plan is in L2 before this CTA ends
}

// ---------------------------------------------------------------------------
// cos and sin of pos * freq, times `scale`. The angle and its reduction to
// [-pi/4, pi/4] around a multiple of pi/2 are fp64 (pi/2 in two pieces), so far
// positions keep their phase; there Taylor's series in fp32 (to r^9 and r^10:
// the first terms left out are below 2^-28).
// ---------------------------------------------------------------------------
__device__ __forceinline__ float2 rotary_cos_sin(int32_t pos, double freq, float scale) {
    const double a = static_cast<double>(pos) * freq;
    const double k = rint(a * 0.63661977236758134308);                     // 2 / pi
    double r = fma(-k, 1.57079632679489655800, a);                        // pi / 2, to fp64
    r = fma(-k, 6.12323399573676603587e-17, r);                          // and the rest of it
    const float x = static_cast<float>(r), x2 = x * x;
    float s = fmaf(x2, 1.f / 362880.f, -1.f / 5040.f);
    s = fmaf(x2, s, 1.f / 120.f);
    s = fmaf(x2, s, -1.f / 6.f);
    s = fmaf(x * x2, s, x);
    float c = fmaf(x2, -1.f / 3628800.f, 1.f / 40320.f);
    c = fmaf(x2, c, -1.f / 720.f);
    c = fmaf(x2, c, 1.f / 24.f);
    c = fmaf(x2, c, -0.5f);
    c = fmaf(x2, c, 1.f);
    const int q = static_cast<int>(static_cast<long long>(k) & 3);       // quarter turns
    const float cc = (q & 1) ? s : c, ss = (q & 1) ? c : s;
    return make_float2((q == 1 || q == 2 ? -cc : cc) * scale, (q & 2 ? -ss : ss) * scale);
}

// One pair turned, in fp32.
__device__ __forceinline__ void turn(float x0, float x1, float2 cs, float *y0, float *y1) {
    *y0 = x0 * cs.x - x1 * cs.y;
    *y1 = x0 * cs.y + x1 * cs.x;
}

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
    static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<float> {
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
};

// n / d and n % d for n < 2^31 by a multiplication: m = ceil(2^(32 + s) / d), 2^s >= d.
struct FastDiv {
    uint32_t d, m, s;
    __host__ __device__ void set(uint32_t div) {
        d = div;
        s = 0;
        while ((1ull << s) < div) ++s;
        m = static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - div)) / div + 1);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const {
        return static_cast<uint32_t>((static_cast<uint64_t>(__umulhi(n, m)) + n) >> s);
    }
};

// ---------------------------------------------------------------------------
// Rotary positions of a [tokens, heads, width] tensor, and of a second one with
// heads of its own, in one launch: channels offset .. offset + rot of every head are
// turned pair by pair, the others copied where the output is another tensor.
// A CTA takes TT tokens x HC heads: its TT * rot / 2 cosines and sines are made
// once, in shared memory, and serve all its heads. A head is `per_head` items:
// 16-byte vectors where strides and widths allow (kVec; in the half layout a
// vector of each half), single pairs and channels otherwise.
// Bound by HBM for prompts (every byte once in and once out), by latency for a
// step's tokens.
// ---------------------------------------------------------------------------
struct RotaryTensor {
    const void *in;
    void *out;
    int64_t in_token, in_head, out_token, out_head;   // strides in elements
};

struct RotaryArgs {
    RotaryTensor x[2];
    const int32_t *positions;    // [tokens]; a row with a negative one is left as it is
    const double *inv_freq;      // [half]
    float mscale, sign;          // sign -1: the inverse turn
    int32_t tokens, heads[2];    // heads[1] = 0: one tensor
    int32_t width, offset, half;
    int32_t TT, HC;              // tokens and heads of a CTA
    FastDiv per_head, per_token;   // items of a head, heads of a CTA
    int32_t turned;              // of them, items that turn pairs
};

constexpr int kRotaryThreads = 256;
constexpr int kRotaryMaxTable = 4096;   // cosine / sine pairs of a CTA (32 KB)

template <typename T, bool kHalf, bool kVec>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const RotaryArgs a) {
    extern __shared__ float2 rotary_cs[];
    constexpr int E = kVec ? 16 / static_cast<int>(sizeof(T)) : 1;
    union Vec {
        uint4 u;
        T e[16 / sizeof(T)];
    };
    const int32_t t0 = blockIdx.x * a.TT, h0 = blockIdx.y * a.HC;
    const int32_t nt = min(a.TT, a.tokens - t0), nh = min(a.HC, a.heads[0] + a.heads[1] - h0);
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    for (int i = threadIdx.x; i < nt * a.half; i += kRotaryThreads) {
        const int t = i / a.half, p = i - t * a.half;
        const float2 cs = rotary_cos_sin(a.positions[t0 + t], a.inv_freq[p], a.mscale);
        rotary_cs[i] = make_float2(cs.x, a.sign * cs.y);
    }
    __syncthreads();
    const uint32_t items = static_cast<uint32_t>(nt) * a.HC * a.per_head.d;
    for (uint32_t i = threadIdx.x; i < items; i += kRotaryThreads) {
        const uint32_t row = a.per_head.div(i), item = i - row * a.per_head.d;
        const uint32_t t = a.per_token.div(row), hh = row - t * a.per_token.d;
        if (static_cast<int32_t>(hh) >= nh || a.positions[t0 + t] < 0) continue;
        int32_t h = h0 + static_cast<int32_t>(hh);
        const int w = h >= a.heads[0] ? 1 : 0;
        h -= w ? a.heads[0] : 0;
        const RotaryTensor &x = a.x[w];
        const T *in = static_cast<const T *>(x.in) + (t0 + t) * x.in_token + h * x.in_head;
        T *out = static_cast<T *>(x.out) + (t0 + t) * x.out_token + h * x.out_head;
        if (static_cast<int32_t>(item) >= a.turned) {   // a channel (vector) that is not turned
            int32_t c = (static_cast<int32_t>(item) - a.turned) * E;
            if (c >= a.offset) c += 2 * a.half;
            if constexpr (kVec) *reinterpret_cast<uint4 *>(out + c) = *reinterpret_cast<const uint4 *>(in + c);
            else out[c] = in[c];
            continue;
        }
        const float2 *cs = rotary_cs + t * a.half;
        if constexpr (kVec && kHalf) {
            const int32_t p = static_cast<int32_t>(item) * E, c = a.offset + p;
            Vec lo, hi;
            lo.u = *reinterpret_cast<const uint4 *>(in + c);
            hi.u = *reinterpret_cast<const uint4 *>(in + c + a.half);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                float y0, y1;
                turn(Elem<T>::get(lo.e[j]), Elem<T>::get(hi.e[j]), cs[p + j], &y0, &y1);
                lo.e[j] = Elem<T>::put(y0);
                hi.e[j] = Elem<T>::put(y1);
            }
            *reinterpret_cast<uint4 *>(out + c) = lo.u;
            *reinterpret_cast<uint4 *>(out + c + a.half) = hi.u;
        } else if constexpr (kVec) {
            const int32_t p = static_cast<int32_t>(item) * (E / 2), c = a.offset + 2 * p;
            Vec v;
            v.u = *reinterpret_cast<const uint4 *>(in + c);
#pragma unroll
            for (int j = 0; j < E / 2; ++j) {
                float y0, y1;
                turn(Elem<T>::get(v.e[2 * j]), Elem<T>::get(v.e[2 * j + 1]), cs[p + j], &y0, &y1);
                v.e[2 * j] = Elem<T>::put(y0);
                v.e[2 * j + 1] = Elem<T>::put(y1);
            }
            *reinterpret_cast<uint4 *>(out + c) = v.u;
        } else {
            const int32_t p = static_cast<int32_t>(item);
            const int32_t c0 = a.offset + (kHalf ? p : 2 * p), c1 = kHalf ? c0 + a.half : c0 + 1;
            float y0, y1;
            turn(Elem<T>::get(in[c0]), Elem<T>::get(in[c1]), cs[p], &y0, &y1);
            out[c0] = Elem<T>::put(y0);
            out[c1] = Elem<T>::put(y1);
        }
    }
}

// ---------------------------------------------------------------------------
// Cache write by slot map: token t's c_KV (copied, or as E4M3 codes with a scale)
// and rotated k_R go to row slots[t] % 64 of page slots[t] / 64; slot -1 is a row of
// a padded batch and is skipped. One warp per token, 16-byte vectors; each lane
// turns the pairs lane, lane + 32, ...
// Bound by HBM: every byte once in and once out.
// ---------------------------------------------------------------------------
struct AppendSlotsArgs {
    const __nv_bfloat16 *ckv_new, *kr_new;
    int64_t ckv_new_stride, kr_new_stride;   // elements between tokens
    const int64_t *slots;                    // [T]
    const int32_t *positions;                // [T], or null: k_R is copied
    const double *inv_freq;                  // [d_r / 2]
    __nv_bfloat16 *ckv;                      // bf16 cache, or null
    uint8_t *ckv8;                           // E4M3 cache
    float *scales;                           // [pages, 64] with it
    __nv_bfloat16 *kr;
    int64_t ckv_page_stride, ckv_token_stride, kr_page_stride, kr_token_stride;   // elements
    float mscale;
    int32_t T, d_c, d_r, num_pages, half_layout;
};

__global__ void __launch_bounds__(256) append_slots_kernel(const AppendSlotsArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    if (t >= a.T) return;
    const int64_t at = a.slots[t];
    if (at < 0 || at >= static_cast<int64_t>(a.num_pages) * 64) {   // uniform over the warp
        if (at != -1 && lane == 0) record_error(kErrDeviceBounds);
        return;
    }
    const int64_t page = at / 64, row = at % 64;
    const __nv_bfloat16 *src = a.ckv_new + t * a.ckv_new_stride;
    if (a.ckv8) {
        const float scale = quantise_row_e4m3(reinterpret_cast<const uint4 *>(src), a.d_c,
                                              a.ckv8 + page * a.ckv_page_stride + row * a.ckv_token_stride, lane);
        if (lane == 0) a.scales[at] = scale;
    } else {
        uint4 *dst = reinterpret_cast<uint4 *>(a.ckv + page * a.ckv_page_stride + row * a.ckv_token_stride);
        for (int i = lane; i < a.d_c / 8; i += 32) dst[i] = reinterpret_cast<const uint4 *>(src)[i];
    }
    const __nv_bfloat16 *r = a.kr_new + t * a.kr_new_stride;
    __nv_bfloat16 *rd = a.kr + page * a.kr_page_stride + row * a.kr_token_stride;
    const int half = a.d_r / 2;
    for (int p = lane; p < half; p += 32) {
        const int c0 = a.half_layout ? p : 2 * p, c1 = a.half_layout ? p + half : 2 * p + 1;
        __nv_bfloat16 y0 = r[c0], y1 = r[c1];
        if (a.positions) {
            const int32_t pos = a.positions[t];
            if (pos < 0 && p == 0) record_error(kErrDeviceBounds);
            float f0, f1;
            turn(__bfloat162float(y0), __bfloat162float(y1), rotary_cos_sin(max(pos, 0), a.inv_freq[p], a.mscale),
                 &f0, &f1);
            y0 = __float2bfloat16_rn(f0);
            y1 = __float2bfloat16_rn(f1);
        }
        rd[c0] = y0;
        rd[c1] = y1;
    }
}

}  // namespace mla
