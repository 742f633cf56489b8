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
// Bound by latency: launch, lengths, a block scan, two dependent loads per token. The
// bytes are 16 a token. 64 drafts of up to 8 tokens: 4.2 us, of up to 64 5.0, of up to 256 (a
// walk of dependent loads up the tree) 6.1; 1024 prompt pieces, 262144 tokens: 7.5 us.
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
constexpr int kPlanMaxDepth = 32 * kPlanMaxWords;   // ancestors that a walk counts

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
    const int64_t big = 0x7FFFFFFF;
    const int64_t cap = min(static_cast<int64_t>(a.max_pages) * 64, big);
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
    // thread i sums `per` consecutive sequences, the block scans the sums, and the thread
    // lays its sequences out from there
    const int32_t per = (a.batch + kPlanThreads - 1) / kPlanThreads;
    const int32_t b_lo = min(tid * per, a.batch), b_hi = min(b_lo + per, a.batch);
    int64_t st = 0, sf = 0;
    for (int32_t b = b_lo; b < b_hi; ++b) {
        int64_t c, n;
        lens(b, &c, &n);
        st += n;
        sf += (c + n + 63) / 64 - (c + 63) / 64;
    }
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
    st -= mt;
    sf -= mf;
    for (int w = 0; w < warp; ++w) {
        st += warp_sum[0][w];
        sf += warp_sum[1][w];
    }
    for (int32_t b = b_lo; b < b_hi; ++b) {
        int64_t c, n;
        lens(b, &c, &n);
        cu[b] = static_cast<int32_t>(min(st, big));
        fresh[b] = static_cast<int32_t>(min(sf, big));
        st += n;
        sf += (c + n + 63) / 64 - (c + 63) / 64;
    }
    if (tid == kPlanThreads - 1) {   // its sums are the totals, whether or not it had sequences
        cu[a.batch] = static_cast<int32_t>(min(st, big));
        fresh[a.batch] = static_cast<int32_t>(min(sf, big));
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
    // (indices are unsigned: a stride past the last of 2^31 - 1 does not wrap)
    const uint32_t first = blockIdx.x * kPlanThreads + tid, stride = gridDim.x * kPlanThreads;

    for (uint32_t t = first; t < static_cast<uint32_t>(a.num_tokens); t += stride) {
        int32_t id = -1, pos = -1;
        int64_t slot = -1;
        uint32_t mask[kPlanMaxWords] = {};
        if (t < static_cast<uint32_t>(total)) {
            id = plan_find(cu, a.batch, t);
            const int32_t i = static_cast<int32_t>(t) - cu[id];
            const int64_t c = a.cached_lens[id], at = c + i;
            const int64_t pg = at / 64 - (c + 63) / 64;
            const int32_t page = pg < 0 ? a.block_table[static_cast<int64_t>(id) * a.max_pages + at / 64]
                                        : fresh_page(fresh[id] + pg);
            if (page >= 0) slot = static_cast<int64_t>(page) * 64 + at % 64;
            else bad = true;
            int32_t depth = i;
            if (a.parents) {
                // up the tree; a parent comes before its child, so this ends. An entry
                // that does not is taken for a root, and a request with more tokens than
                // any tree (reported) may hold chains without a bound: their walks end early.
                const int32_t *par = a.parents + cu[id];
                depth = 0;
                for (int32_t j = i; depth < kPlanMaxDepth;) {
#pragma unroll
                    for (int w = 0; w < kPlanMaxWords; ++w) mask[w] |= (j >> 5) == w ? 1u << (j & 31) : 0u;
                    const int32_t up = par[j];
                    if (up >= j) bad = true;
                    if (up < 0 || up >= j) break;
                    j = up;
                    ++depth;
                }
                if (i >= a.max_nodes) {
                    bad = true;
#pragma unroll
                    for (int w = 0; w < kPlanMaxWords; ++w)
                        if (32 * w + 31 >= a.max_nodes)
                            mask[w] &= 32 * w >= a.max_nodes ? 0u : (1u << (a.max_nodes & 31)) - 1u;
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
    for (uint32_t u = first; u < static_cast<uint32_t>(pages); u += stride) {
        const int32_t k = static_cast<int32_t>(u), b = plan_find(fresh, a.batch, k);
        const int64_t p0 = (static_cast<int64_t>(a.cached_lens[b]) + 63) / 64;
        a.block_table[static_cast<int64_t>(b) * a.max_pages + p0 + (k - fresh[b])] = fresh_page(k);
    }
    for (int32_t b = static_cast<int32_t>(first); b <= a.batch; b += static_cast<int32_t>(stride)) {
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
// [-pi/4, pi/4] around a multiple of pi/2 are fp64 (pi/2 in two pieces, the method of
// Cody and Waite), so far positions keep their phase; there Taylor's series in fp32 (to r^9 and r^10:
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

// ---------------------------------------------------------------------------
// Rotary positions of a [tokens, heads, width] tensor, and of a second one with
// heads of its own, in one launch: channels offset .. offset + rot of every head are
// turned pair by pair, the others copied where the output is another tensor.
// A thread has one place of a token's rows (a head's vector of 16 bytes; in the half
// layout one of each half, or two copied ones (290 us below with one); where strides or widths
// do not allow that (kVec), a pair or a channel) and walks TT tokens with it, the loads of four
// of them in flight, so no index is divided in the loop; a CTA's up to 256 places share the
// TT * rot / 2 cosines and sines, made while the first loads are on their way. The CTAs of
// a row have equal shares of its places, not 256 and a rest (4096 tokens x 4 heads of 128 fp32:
// 3.8 us, not 8.1).
// Bound by HBM for prompts (every byte once in and once out), by latency for a
// step's tokens. 16384 tokens x 129 heads of 192, 64 of them turned: 259 us, 6.3 TB/s (255 us interleaved).
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
    int32_t TT;                  // tokens of a CTA
    int32_t turned, copied;      // places of a head that turn, and that copy
};

constexpr int kRotaryThreads = 256;
constexpr int kRotaryMaxTable = 4096;   // cosine / sine pairs of a CTA (32 KB)
constexpr int kRotaryMaxTokens = 32;    // tokens of a CTA
constexpr int kRotaryFlight = 4;

template <typename T, bool kHalf, bool kVec>
__global__ void __launch_bounds__(kRotaryThreads, kVec && !kHalf ? 5 : 3) rotary_kernel(const RotaryArgs a) {
    extern __shared__ float2 rotary_cs[];
    __shared__ int32_t s_pos[kRotaryMaxTokens];
    constexpr int E = kVec ? 16 / static_cast<int>(sizeof(T)) : 1;
    constexpr int U = kRotaryFlight;
    union Vec {
        uint4 u;
        T e[16 / sizeof(T)];
    };
    const int32_t t0 = blockIdx.x * a.TT, nt = min(a.TT, a.tokens - t0);
    // this thread's place: head h of both tensors' and channel c
    const int32_t n = blockIdx.y * blockDim.x + threadIdx.x, per_head = a.turned + a.copied;
    int32_t h = n / per_head;
    const int32_t place = n - h * per_head;
    const bool active = h < a.heads[0] + a.heads[1];
    if (!active) h = 0;
    // kHalf: the turned places, then the copied vectors, two a place as well; else copied
    // channels before the turned ones, those, and the copied ones after
    const int32_t before = a.copied && !kHalf ? a.offset / E : 0;
    const bool turns = place >= before && place < before + a.turned;
    const int32_t item = place - before;
    auto copied = [&](int32_t j) { return j * E < a.offset ? j * E : j * E + 2 * a.half; };   // channel of the j-th
    const int32_t c = turns            ? a.offset + item * (kHalf || kVec ? E : 2)
                      : kHalf          ? copied(item - a.turned)
                      : place < before ? place * E
                                       : a.offset + 2 * a.half + (item - a.turned) * E;
    const int w = h >= a.heads[0] ? 1 : 0;
    const RotaryTensor &x = a.x[w];
    h -= w ? a.heads[0] : 0;
    const T *in = static_cast<const T *>(x.in) + static_cast<int64_t>(t0) * x.in_token + h * x.in_head + c;
    T *out = static_cast<T *>(x.out) + static_cast<int64_t>(t0) * x.out_token + h * x.out_head + c;
    const int64_t in_token = x.in_token, out_token = x.out_token;
    // a second vector: the pair's other half, or another copied one
    const int32_t next = item - a.turned + a.copied;
    const bool two = turns ? kHalf || !kVec : kHalf && next * E < a.width - 2 * a.half;
    const int32_t apart = !kHalf ? 1 : turns ? a.half : copied(next) - c;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    Vec lo[U], hi[U];
    auto fetch = [&](int32_t t) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!active || t + u >= nt) break;
            const T *p = in + (t + u) * in_token;
            if constexpr (kVec) {
                lo[u].u = *reinterpret_cast<const uint4 *>(p);
                if (two) hi[u].u = *reinterpret_cast<const uint4 *>(p + apart);
            } else {
                lo[u].e[0] = p[0];
                if (two) hi[u].e[0] = p[apart];
            }
        }
    };
    fetch(0);
    for (int i = threadIdx.x; i < nt; i += blockDim.x) s_pos[i] = a.positions[t0 + i];
    for (int i = threadIdx.x; i < nt * a.half; i += blockDim.x) {
        const int t = i / a.half, p = i - t * a.half;
        const float2 cs = rotary_cos_sin(a.positions[t0 + t], a.inv_freq[p], a.mscale);
        rotary_cs[i] = make_float2(cs.x, a.sign * cs.y);
    }
    __syncthreads();
    if (!active) return;
    const float2 *cs0 = rotary_cs + item * (kVec && !kHalf ? E / 2 : E);
    for (int32_t t = 0; t < nt; t += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u >= nt) break;
            if (s_pos[t + u] < 0) continue;   // a skipped row
            T *q = out + (t + u) * out_token;
            if (turns) {
                const float2 *cs = cs0 + (t + u) * a.half;
                if constexpr (kVec && !kHalf) {
#pragma unroll
                    for (int j = 0; j < E / 2; ++j) {
                        float y0, y1;
                        turn(Elem<T>::get(lo[u].e[2 * j]), Elem<T>::get(lo[u].e[2 * j + 1]), cs[j], &y0, &y1);
                        lo[u].e[2 * j] = Elem<T>::put(y0);
                        lo[u].e[2 * j + 1] = Elem<T>::put(y1);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < E; ++j) {
                        float y0, y1;
                        turn(Elem<T>::get(lo[u].e[j]), Elem<T>::get(hi[u].e[j]), cs[j], &y0, &y1);
                        lo[u].e[j] = Elem<T>::put(y0);
                        hi[u].e[j] = Elem<T>::put(y1);
                    }
                }
            }
            if constexpr (kVec) {
                *reinterpret_cast<uint4 *>(q) = lo[u].u;
                if (two) *reinterpret_cast<uint4 *>(q + apart) = hi[u].u;
            } else {
                q[0] = lo[u].e[0];
                if (two) q[apart] = hi[u].e[0];
            }
        }
        fetch(t + U);
    }
}

// ---------------------------------------------------------------------------
// Cache write by slot map: token t's c_KV (copied, or as E4M3 codes with a scale)
// and rotated k_R go to row slots[t] % 64 of page slots[t] / 64; slot -1 is a row of
// a padded batch and is skipped. One warp per token; its row (up to 512 channels),
// slot, position and key are requested together, before any of them is looked at.
// The bytes are every one once in and once out; a warp has one token and ends, so nothing of
// a next one is in flight while a row's maximum, division and conversion run: 32768 tokens to
// E4M3 take 13.6 us, 4.3 TB/s; a step's 128 tokens 1.5 us.
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

// 16 bytes of a row that is read once.
__device__ __forceinline__ uint4 ld_row(const __nv_bfloat16 *row, int i) {
    return __ldcs(reinterpret_cast<const uint4 *>(row) + i);
}

__global__ void __launch_bounds__(256) append_slots_kernel(const AppendSlotsArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    if (t >= a.T) return;
    const __nv_bfloat16 *src = a.ckv_new + t * a.ckv_new_stride;
    const __nv_bfloat16 *kr = a.kr_new + t * a.kr_new_stride;
    const int half = a.d_r / 2;
    // pair lane of the key: channels c0 and c1
    const int c0 = a.half_layout ? lane : 2 * lane, c1 = a.half_layout ? lane + half : 2 * lane + 1;
    const int64_t at = a.slots[t];
    const int32_t pos = a.positions ? a.positions[t] : 0;
    uint4 v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        v[i] = lane + 32 * i < a.d_c / 8 ? ld_row(src, lane + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
    __nv_bfloat16 k0 = __float2bfloat16_rn(0.f), k1 = k0;
    double freq = 0.0;
    if (lane < half) {
        k0 = kr[c0];
        k1 = kr[c1];
        if (a.positions) freq = a.inv_freq[lane];
    }
    if (at < 0 || at >= static_cast<int64_t>(a.num_pages) * 64) {   // uniform over the warp
        if (at != -1 && lane == 0) record_error(kErrDeviceBounds);
        return;
    }
    if (a.positions && pos < 0 && lane == 0) record_error(kErrDeviceBounds);
    const int64_t page = at / 64, row = at % 64;
    if (a.ckv8) {
        uint8_t *dst = a.ckv8 + page * a.ckv_page_stride + row * a.ckv_token_stride;
        const float scale = a.d_c <= 512 ? quantise_row_e4m3(v, a.d_c, dst, lane)
                                         : quantise_row_e4m3(reinterpret_cast<const uint4 *>(src), a.d_c, dst, lane);
        if (lane == 0) a.scales[at] = scale;
    } else {
        uint4 *dst = reinterpret_cast<uint4 *>(a.ckv + page * a.ckv_page_stride + row * a.ckv_token_stride);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (lane + 32 * i < a.d_c / 8) dst[lane + 32 * i] = v[i];
        for (int i = lane + 64; i < a.d_c / 8; i += 32) dst[i] = ld_row(src, i);
    }
    __nv_bfloat16 *rd = a.kr + page * a.kr_page_stride + row * a.kr_token_stride;
    for (int p = lane; p < half; p += 32) {
        const int d0 = a.half_layout ? p : 2 * p, d1 = a.half_layout ? p + half : 2 * p + 1;
        if (p > lane) {   // keys wider than 64
            k0 = kr[d0];
            k1 = kr[d1];
            if (a.positions) freq = a.inv_freq[p];
        }
        if (a.positions) {
            float f0, f1;
            turn(__bfloat162float(k0), __bfloat162float(k1), rotary_cos_sin(max(pos, 0), freq, a.mscale), &f0, &f1);
            k0 = __float2bfloat16_rn(f0);
            k1 = __float2bfloat16_rn(f1);
        }
        rd[d0] = k0;
        rd[d1] = k1;
    }
}

}  // namespace mla
