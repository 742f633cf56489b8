/*
 * mla_step.h -- a step with any number of query tokens per sequence over the
 * paged latent cache: a draft (chain or tree) that a target model verifies in
 * one pass, or short prompt pieces. Four operators, used in this order:
 *     mla_step_plan           pages, slots, positions and tree masks from the request lengths
 *     mla_rotary              rotary positions of the new queries (and keys)
 *     mla_append_kv_slots     the new tokens' c_KV and k_R into the cache, by slot map
 *     mla_decode_tree         attention of every new token to its sequence's cache
 * with mla_absorb_q before and mla_absorb_out after mla_decode_tree, as in a
 * decode step.
 *
 * The conventions of mla_decode.h hold for every call: device pointers unless a
 * parameter says "host", nothing allocated, asynchronous on `stream`, argument
 * errors returned before anything is launched, data errors in the device error
 * word, deterministic results. mla_decode_tree reads seq_lens, cu_tokens and
 * block_table before its dependency wait, as the decode calls do: a custom kernel that
 * lets its dependents start early must not write them directly before it.
 *
 * Packed tokens: the step's query tokens lie sequence after sequence; sequence b
 * owns rows cu_tokens[b] .. cu_tokens[b + 1) of every per-token tensor, its newest
 * n_b = cu_tokens[b + 1] - cu_tokens[b] tokens. Per-token tensors may have more
 * rows than cu_tokens[batch] (a captured step of fixed size): rows behind the
 * last sequence are skipped, and outputs there are left as they were except where
 * a call says what it writes.
 */
#ifndef MLA_STEP_H
#define MLA_STEP_H

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MLA_STEP_MAX_BATCH 16384   /* requests of one mla_step_plan */
#define MLA_TREE_MAX_NODES 256     /* query tokens per sequence; above it the decompress branch is cheaper */

/*
 * Plan of a step on the GPU, without a host round trip. Request b has
 * cached_lens[b] tokens in the cache and adds new_lens[b] (0: an idle row).
 *   seq_lens[b]  = cached_lens[b] + new_lens[b]
 *   cu_tokens[b] = sum of new_lens before b                       ([batch + 1])
 *   block_table[b][p], ceil(cached / 64) <= p < ceil(seq_len / 64), is set to the
 *       next page of free_pages, from free_pages[*free_head] on, requests in order;
 *       all other entries are left as they were
 *   free_head_out = *free_head + pages taken
 * and for token t = cu_tokens[b] + i:
 *   seq_ids[t]   = b
 *   positions[t] = cached_lens[b] + depth(i)         (rotary position)
 *   slots[t]     = block_table[b][(cached + i) / 64] * 64 + (cached + i) % 64
 * Without parents (NULL) depth(i) = i. With parents [num_tokens], parents[t] is
 * the index (within the request) of the drafted token that token t follows, which
 * must come before it, or negative for a child of the context: depth counts the
 * ancestors, and masks[t] ([num_tokens, ceil(max_nodes / 32)] words, bit j of
 * word w: token 32 w + j) marks the token itself and its ancestors. max_nodes
 * (1 .. MLA_TREE_MAX_NODES) bounds new_lens then; without parents it is ignored
 * and masks is not written.
 * Rows t >= cu_tokens[batch] get seq_ids -1, positions -1, slots -1, masks 0.
 * A request whose lengths are negative or do not fit its table row is planned with
 * no new tokens; a token without a page (the free list ran out, or a negative old
 * table entry) gets slot -1, a table entry without one -1; a parent that does not
 * come before its child counts as none; tokens beyond num_tokens are not written;
 * of a request with more than max_nodes tokens, mask bits beyond max_nodes are
 * dropped and depths end at MLA_TREE_MAX_NODES. All of these set
 * MLA_ERR_DEVICE_BOUNDS.
 * After a step of which not every token is kept, cached_lens[b] of the next plan ends where the
 * kept tokens still lie one after the other (those of a tree's path that do not are written again,
 * as new tokens). The pages past it, entries ceil(cached / 64) .. ceil(seq_len / 64) of the row, are the
 * caller's to put back on the free list first: the next plan takes fresh ones for them.
 * batch <= MLA_STEP_MAX_BATCH (else MLA_ERR_UNSUPPORTED). Outputs must not
 * overlap inputs; in particular free_head_out and free_head are different words.
 * batch = 0 writes the padded rows, cu_tokens[0] = 0 and free_head_out.
 */
mla_status mla_step_plan(const int32_t *cached_lens, const int32_t *new_lens, int32_t batch,
                         const int32_t *free_pages, int32_t num_free, const int32_t *free_head,
                         int32_t *block_table, int32_t max_pages_per_seq, const int32_t *parents,
                         int32_t max_nodes, int32_t num_tokens, int32_t *seq_lens,
                         int32_t *cu_tokens, int32_t *seq_ids, int32_t *positions, int64_t *slots,
                         uint32_t *masks, int32_t *free_head_out, void *stream);

/* Rotary frequencies in fp64, computed on the host: inv_freq [rot_dim / 2]
 * (host) and *mscale (host), the factor on cosines and sines. With
 * f_i = theta^(-2 i / rot_dim):
 *   NONE    f_i, 1
 *   LINEAR  f_i / factor, 1                  (position interpolation)
 *   NTK     f_i of the base theta * factor^(rot_dim / (rot_dim - 2)), 1
 *   YARN    f_i / factor * r_i + f_i (1 - r_i), 0.1 ln(factor) + 1  (factor > 1)
 *           with the ramp r_i = clamp((i - lo) / max(hi - lo, 0.001), 0, 1),
 *           lo = max(floor(n(beta_fast)), 0), hi = min(ceil(n(beta_slow)), rot_dim - 1),
 *           n(b) = rot_dim ln(original_max / (2 pi b)) / (2 ln theta)
 * (NTK by parts and its attention factor as published for YaRN.) theta > 1,
 * factor >= 1, rot_dim even and positive; original_max, beta_fast and beta_slow > 0
 * matter for YARN only; NTK needs rot_dim > 2. */
typedef enum {
    MLA_ROPE_NONE = 0,
    MLA_ROPE_LINEAR = 1,
    MLA_ROPE_NTK = 2,
    MLA_ROPE_YARN = 3
} mla_rope_scaling;
mla_status mla_rope_frequencies(int32_t rot_dim, double theta, int32_t scaling, double factor,
                                double original_max, double beta_fast, double beta_slow,
                                double *inv_freq, double *mscale);

typedef enum { MLA_BF16 = 0, MLA_FP16 = 1, MLA_FP32 = 2 } mla_dtype;
typedef enum {
    MLA_ROPE_INTERLEAVED = 0,   /* pairs (2i, 2i + 1): mla_absorb_q_rope's and mla_append_kv's */
    MLA_ROPE_HALF = 1           /* pairs (i, i + rot_dim / 2) */
} mla_rope_layout;

/* One [tokens, heads, width] tensor (host struct): element (t, h, c) is at
 * in[t * in_token + h * in_head + c], and the result's at out[...] likewise
 * (strides in elements; the channels of a head are contiguous; in strides may be
 * 0, out strides of more than one token or head may not). out == in with the same strides
 * turns in place; otherwise the two must not overlap. */
typedef struct {
    const void *in;
    void *out;
    int64_t in_token, in_head, out_token, out_head;
    int32_t heads;
} mla_rotary_tensor;

/*
 * Rotary positions. In every head of x (and of y, a second tensor with heads of
 * its own, e.g. the keys; NULL: none) channel pair i of channels
 * offset .. offset + rot_dim turns by a = positions[t] * inv_freq[i]:
 *   y0 = mscale (x0 cos a - x1 sin a),   y1 = mscale (x0 sin a + x1 cos a)
 * with the angle and its reduction in fp64 and the rotation in fp32, rounded once to
 * `dtype`. The other channels are copied (in place: left alone). inverse != 0
 * turns by -a (with the same mscale): the transpose, i.e. the gradient of x given
 * y's, and with mscale 1 the way back. Rows with a negative position are skipped (their output is left as it was).
 * inv_freq [rot_dim / 2] fp64 and positions [num_tokens] int32 are device
 * pointers. rot_dim even, 2 <= rot_dim <= 4096, 0 <= offset, offset + rot_dim <= width <= 65536,
 * heads of both tensors together <= 65536, and heads * width <= 2^24
 * (MLA_ERR_UNSUPPORTED beyond); any strides (16-byte accesses are used where pointers,
 * strides and widths are multiples of 16 bytes).
 */
mla_status mla_rotary(const mla_rotary_tensor *x, const mla_rotary_tensor *y, int32_t dtype,
                      int32_t num_tokens, int32_t width, int32_t offset, int32_t rot_dim,
                      const int32_t *positions, const double *inv_freq, float mscale,
                      int32_t layout, int32_t inverse, void *stream);

/*
 * Cache write by slot map: for each token t with slot s = slots[t] >= 0
 *   c_KV pool [s / 64][s % 64][:] = ckv_new[t, :]                       (bit copy)
 *   k_R  pool [s / 64][s % 64][:] = mla_rotary of kr_new[t, :] at positions[t]
 * Slot -1 is skipped (a row of a padded batch); any other slot outside the pool is
 * skipped and sets MLA_ERR_DEVICE_BOUNDS. positions == NULL copies k_R. Unlike
 * mla_append_kv, the rotary position is independent of the cache slot, as the
 * tokens of a draft tree need. Slots of one call must differ; every other row of
 * the pools is left untouched. A negative position is treated as 0 and sets
 * MLA_ERR_DEVICE_BOUNDS.
 * ckv_new [T, d_latent], kr_new [T, d_rope] bf16 with token strides in elements
 * (the two may be views of one [T, d_latent + d_rope] tensor); ckv_new 16-byte
 * aligned with a stride that is a multiple of 8. Pools as for mla_append_kv.
 */
mla_status mla_append_kv_slots(const mla_dims *dims, const void *ckv_new, int64_t ckv_new_stride,
                               const void *kr_new, int64_t kr_new_stride, const int64_t *slots,
                               const int32_t *positions, const double *inv_freq, float mscale,
                               int32_t layout, int32_t num_tokens, const mla_pool *ckv,
                               const mla_pool *kr, int32_t num_pages, void *stream);

/* The same into the E4M3 cache, with the quantisation of mla_append_kv_fp8. */
mla_status mla_append_kv_slots_fp8(const mla_dims *dims, const void *ckv_new,
                                   int64_t ckv_new_stride, const void *kr_new,
                                   int64_t kr_new_stride, const int64_t *slots,
                                   const int32_t *positions, const double *inv_freq, float mscale,
                                   int32_t layout, int32_t num_tokens, const mla_pool *ckv8,
                                   float *scales, const mla_pool *kr, int32_t num_pages,
                                   void *stream);

/* Partitions mla_decode_tree should be given on a device with num_sms
 * multiprocessors (one per CTA pair for d_latent 512, one per CTA for 64), and the
 * bytes of workspace that num_parts partitions need: 2 num_parts slots of 128
 * query rows and num_parts notes of 16 bytes, whatever the batch. Host only; 0 for invalid arguments. */
int32_t mla_tree_num_parts(const mla_dims *dims, int32_t num_sms);
size_t mla_tree_workspace_bytes(const mla_dims *dims, int32_t num_parts);

/*
 * Attention of a step's packed query tokens over the paged latent cache, in
 * latent space. Token t = cu_tokens[b] + i of sequence b, head h:
 *   s[u]  = scale * (q[t, h, 0:d_c] . c_KV[u] + q[t, h, d_c:] . k_R[u])
 *   o_lat[t, h, :] = bf16( sum_u softmax(s)_u c_KV[u] ),   lse_out[t, h] = log sum_u exp(s[u])
 * over the tokens u of the sequence that t sees: every context token
 * (u < seq_lens[b] - n_b) and drafted token seq_lens[b] - n_b + j where bit j of
 * masks[t] is set; masks == NULL is a chain, j <= i. A row that sees nothing gives
 * 0 and -inf. What a row does not see does not reach it, whatever it holds: NaN and
 * infinities in the cache past a sequence's end, and in the latent or key of a
 * drafted token that its mask leaves out, included. (A visible token whose score is -inf
 * has weight 0; a visible NaN or +inf score makes the row NaN.)
 *   q           [num_tokens, H, d_c + d_R] bf16 (the q_out of mla_absorb_q), 16-byte aligned
 *   block_table, seq_lens, pools: as for mla_decode_splitkv; seq_lens counts the
 *               n_b new tokens, which are already in the cache
 *   cu_tokens   [batch + 1] int32; n_b = 0 is allowed (nothing is done for b)
 *   masks       [num_tokens, ceil(max_nodes / 32)] words, or NULL
 *   max_nodes   an upper bound of every n_b, 1 .. MLA_TREE_MAX_NODES (host)
 *   workspace   >= mla_tree_workspace_bytes(dims, num_parts), 256-byte aligned; written before
 *               it is read by the same call. Calls that may overlap need one each.
 *   o_lat       [num_tokens, H, d_c] bf16, lse_out [num_tokens, H] fp32 (may be NULL)
 * dims->n_q is ignored; num_heads <= 128. A sequence whose length does not fit its
 * table row, or with more tokens than max_nodes, than its length or than q has
 * rows, is skipped and sets MLA_ERR_DEVICE_BOUNDS, as a page id outside
 * [0, num_pages) does; a step whose sequences hold more than num_tokens tokens together
 * (a cu_tokens that turns back) is skipped as a whole. Deterministic for a given num_parts.
 * num_tokens * num_heads and the plan's cost must stay below 2^31, max_pages_per_seq below
 * 2^25 - 1 (MLA_ERR_UNSUPPORTED): (num_tokens * num_heads / 64 + batch) * (max_pages_per_seq + 16).
 */
mla_status mla_decode_tree(const mla_dims *dims, const void *q, int32_t num_tokens,
                           const mla_pool *ckv, const mla_pool *kr, int32_t num_pages,
                           const int32_t *block_table, int32_t max_pages_per_seq,
                           const int32_t *seq_lens, const int32_t *cu_tokens, int32_t batch,
                           const uint32_t *masks, int32_t max_nodes, int32_t num_parts,
                           void *workspace, size_t workspace_bytes, void *o_lat, float *lse_out,
                           void *stream);

/* The same over the E4M3 cache (d_latent 512 only), each c_KV element dequantised
 * as in mla_decode_splitkv_fp8. */
mla_status mla_decode_tree_fp8(const mla_dims *dims, const void *q, int32_t num_tokens,
                               const mla_pool *ckv8, const float *scales, const mla_pool *kr,
                               int32_t num_pages, const int32_t *block_table,
                               int32_t max_pages_per_seq, const int32_t *seq_lens,
                               const int32_t *cu_tokens, int32_t batch, const uint32_t *masks,
                               int32_t max_nodes, int32_t num_parts, void *workspace,
                               size_t workspace_bytes, void *o_lat, float *lse_out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_STEP_H */
