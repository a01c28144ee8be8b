/*
 * kda_attention.h — C ABI of the operators of a softmax-attention layer, which models place between the
 * recurrent layers of kda.h, for NVIDIA GB300 (sm_103a), in the same library:
 *
 *   kda_qk_norm_*    the norms of queries and keys per head and the position rotation, in one
 *                    pass, with the gradient; for single tokens (kda_qk_norm_step) with the write of
 *                    keys and values into the cache in the same launch
 *   kda_kv_cache_*   writing a paged key-value cache (in the type of the data, or 8-bit with
 *                    one power of two per row) and reading it back
 *   kda_attn_step    the attention of the next tokens of each sequence over that cache
 *
 * Common to all calls, as in kda_mixer.h: tensor pointers are DEVICE pointers of the current device; data
 * tensors are bf16 or fp32 (`dtype`, KDA_DTYPE_*), weights fp32; sums, norms and softmax statistics are
 * held in fp32 and a result is rounded to its tensor's type once. Calls are asynchronous on `stream`,
 * thread-safe, and the same inputs give bitwise equal outputs (no atomics on outputs). Outputs must not
 * alias an input unless stated. Packed sequences: cu_seqlens != NULL holds B + 1 device int32
 * offsets of B sequences in T rows; a malformed array leaves the outputs undefined, touches no memory
 * outside the tensors, and raises KDA_DEVICE_ERR_SEQLENS (kda_get_device_error). Empty sequences and
 * T == 0 are valid.
 *
 * Token strides: `*_stride` is the distance in elements between consecutive tokens of an input (all
 * tokens evenly spaced, the heads and channels of a token contiguous), so that q, k and v may be slices
 * of one projection's output; 0 means contiguous. Outputs are contiguous. Pointers are aligned to
 * their element type unless stated; where all rows are aligned for it, 16 bytes are moved at a time.
 *
 * Errors: as in kda.h; nothing is launched when a status other than KDA_OK or KDA_ERR_CUDA is
 * returned.
 */
#ifndef KDA_ATTENTION_H
#define KDA_ATTENTION_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_DTYPE_E4M3 2 /* a cache's values only */

/* Device-side error bit (kda_get_device_error): a length below 0 or above max_pages * page_size (it
 * is taken as the nearest allowed one), or a page outside [0, pages) where a token lies (the token
 * is not written; the attention and the read-back take it as zeros). */
#define KDA_DEVICE_ERR_CACHE 4

/*
 * kda_kv_cache — a paged cache of keys and values and where the sequences lie in it.
 *
 *   k, v        [pages, heads, page_size, D]: token p of sequence b is row p % page_size of page
 *               block_table[b][p / page_size]. `dtype`: the type of the data, or KDA_DTYPE_E4M3.
 *               16-byte aligned, D a multiple of 16, at most 256; page_size of any size.
 *   k_scale,    [pages, heads, page_size] bytes, KDA_DTYPE_E4M3 only: a row holds the values
 *   v_scale     e4m3 * 2^(byte - 127), byte 1 to 254 (another one leaves results of its own
 *               sequence undefined, not those of others).
 *   page_stride, scale_stride  elements between consecutive pages of k and v, and of the
 *               scales (k and v alike; 0: contiguous). page_stride is a multiple of D.
 *   block_table [B, max_pages] int32, rows table_stride apart (0: max_pages). Entries beyond a
 *               sequence's length are not read. Sequences may share pages that are only read.
 *   lens        [B] int32: the length of each sequence WITH the new tokens of the call: of n new
 *               tokens, token i stands at position lens[b] - n + i. A token at a negative
 *               position is not there (a sequence at rest in a batch has length 0).
 * Rows of a cache number at most 2^31 (page_stride / D times pages). Sequences longer than 2^31 - 65 are taken as long as that.
 */
typedef struct kda_kv_cache {
    void *k, *v;
    uint8_t *k_scale, *v_scale;
    int64_t page_stride, scale_stride;
    int pages, heads, page_size, D, dtype;
    const int32_t *block_table;
    int max_pages;
    int64_t table_stride;
    const int32_t *lens;
} kda_kv_cache;

/*
 * kda_qk_norm_fwd — per row (a token's head) of q and of k:
 *
 *     n = x / sqrt(mean(x^2) + eps) * weight           (n = x without weight)
 *     y = n with pairs (a, b) of its first R channels turned by the token's angle:
 *         (a cos - b sin, b cos + a sin), the other D - R channels as they are
 *
 * Pair i is channels (i, i + R / 2), or (2 i, 2 i + 1) with `interleaved`. Its angle is
 * position * freq[i], freq in units of 2^-64 turns: their product modulo one turn is exact for every
 * position, and cosine and sine are computed from it in fp32.
 *   q, q_out [B, T, q_heads, D], k, k_out [B, T, k_heads, D] `dtype`; q_weight, k_weight [D]
 *   fp32 or NULL; freq [R / 2] (NULL with R == 0); positions [B, T] int32, or NULL: the token's index in
 *   its sequence. 1 <= D <= 256, R even, R <= D. q_out may be q and k_out may be k when they are
 *   contiguous. B times T (packed: T) times (q_heads + 2 k_heads) is below 2^31 - 2^16.
 */
typedef struct kda_qk_norm_params {
    const void *q, *k;
    const float *q_weight, *k_weight;
    const int64_t *freq;
    const int32_t *positions;
    void *q_out, *k_out;
    int64_t q_stride, k_stride;
    int B, T, q_heads, k_heads, D, R;
    const int32_t *cu_seqlens;
    float eps;
    int dtype, interleaved;
} kda_qk_norm_params;

int kda_qk_norm_fwd(const kda_qk_norm_params *p, cudaStream_t stream);

/* kda_qk_norm_bwd — gradients of sum(dq_out * q_out) + sum(dk_out * k_out) for the forward pass `f`
 * (its q_out and k_out are not read): dq, dk like q_out, k_out; dq_weight, dk_weight [D] fp32 (NULL:
 * not wanted; must be NULL without the weight). dq may be dq_out, dk may be dk_out. Scratch:
 * kda_qk_norm_bwd_workspace bytes, as in kda_mixer.h (workspace == NULL: the library's pool). */
typedef struct kda_qk_norm_bwd_params {
    kda_qk_norm_params f;
    const void *dq_out, *dk_out;
    void *dq, *dk;
    float *dq_weight, *dk_weight;
    void *workspace;
    size_t workspace_bytes;
} kda_qk_norm_bwd_params;

int kda_qk_norm_bwd(const kda_qk_norm_bwd_params *p, cudaStream_t stream);
size_t kda_qk_norm_bwd_workspace(const kda_qk_norm_bwd_params *p);

/*
 * kda_qk_norm_step — kda_qk_norm_fwd on the new tokens of the cache's sequences, with k after norm and
 * rotation and v [B, T, k_heads, D] as it is written into the cache as by kda_kv_cache_write
 * (an 8-bit cache takes them from fp32). f.k_out may be NULL (or k, as in kda_qk_norm_fwd). Positions are those in the cache unless
 * f.positions says otherwise (for the rotation alone). Rows of q whose token is not there are
 * computed like the others.
 */
typedef struct kda_qk_norm_step_params {
    kda_qk_norm_params f;
    const void *v;
    int64_t v_stride;
    kda_kv_cache cache;
} kda_qk_norm_step_params;

int kda_qk_norm_step(const kda_qk_norm_step_params *p, cudaStream_t stream);

/*
 * kda_kv_cache_write — the new tokens k, v [B, T, heads, D] `dtype` into the cache, each at its
 * position. An 8-bit cache holds, of a row x, the values e4m3(x 2^-e) (round to nearest even) with the
 * least e >= -126 that leaves the largest finite |x| at 448 or below, and the byte e + 127. (A
 * power of two costs an 8-bit floating-point value no precision, and every product with it is
 * exact.) NaN is kept; a row with an infinity has e = 120 and holds it as 448 * 2^120, beside which numbers below 2^110
 * are zeros. kda_kv_cache_read gives infinity for that, as for all that passes its type (from 248 * 2^120 on); the attention
 * counts it as the number that it is. Otherwise the cache has the type
 * of the data and holds it unchanged. No two tokens of a call may lie in the same place; other
 * places of the cache are left as they were. 2 B T heads (packed: 2 T heads) is below 2^31 - 2^16, here and in
 * kda_kv_cache_read.
 */
typedef struct kda_kv_cache_write_params {
    const void *k, *v;
    int64_t k_stride, v_stride;
    int B, T;
    const int32_t *cu_seqlens;
    int dtype;
    kda_kv_cache cache;
} kda_kv_cache_write_params;

int kda_kv_cache_write(const kda_kv_cache_write_params *p, cudaStream_t stream);

/* kda_kv_cache_read — the reverse: the last T tokens of each sequence (packed: as many as
 * cu_seqlens says) into k, v [B, T, heads, D] `dtype`; zeros for a token that is not there. An
 * 8-bit cache is read into bf16 or fp32 (exactly, within the type's range), another one into its own type. */
typedef struct kda_kv_cache_read_params {
    void *k, *v;
    int B, T;
    const int32_t *cu_seqlens;
    int dtype;
    kda_kv_cache cache;
} kda_kv_cache_read_params;

int kda_kv_cache_read(const kda_kv_cache_read_params *p, cudaStream_t stream);

/*
 * kda_attn_step — attention of the next T tokens (typically one) of each of B sequences over the cache,
 * in which they already lie: for token t of sequence b and query head h, over the positions
 * j < n = lens[b] - T + t + 1 and the key head h / (q_heads / heads),
 *
 *     o = sum_j softmax_j(scale q . k_j) v_j,    lse = log sum_j exp(scale q . k_j)
 *
 * n <= 0 (or scores that are all -infinity): o = 0, lse = -infinity. What lies in the cache at other
 * positions, NaN and infinities too, has no part in the result: with something else there it is the same bit for bit.
 *   q, o [B, T, q_heads, D] `dtype`, q 16-byte aligned with q_stride a multiple of 16 bytes; lse
 *   [B, T, q_heads] fp32 or NULL. The cache has the type of the data or is 8-bit.
 * bf16 data: products of bf16 (the probabilities are rounded to it) summed in fp32; over an 8-bit cache products of fp16, in
 * which its values are exact: a probability times its value's power of two has 11 bits, fewer below 2^-20 of the row's
 * largest and none below 2^-31. fp32 data: fp32 throughout. The values are summed before the division: results are finite for
 * values below 2^89. An infinity in an 8-bit cache that a token sees counts as 1.75 * 2^128: as a value it makes its channel
 * infinite or that large times its probability, and beside it the other channels lose, for bf16 data, what lies 2^31 below; as a
 * key it has all of the weight or none, or makes the row NaN.
 * The sequences' lengths are cut into equal shares for the GPU's SMs, and results of sequences that were
 * cut are joined in the order of their shares: which are cut follows from the lengths and sizes alone.
 * One call reads the cache ceil(T q_heads / heads / 64) times (bf16, D up to 128; 32 for wider heads; fp32
 * 8): T in the hundreds works but is not what it is made for.
 * Limits: q_heads / heads at most 256, T times that below 2^24, B T q_heads below 2^31; the sequences' units of 16 or 32 keys
 * (8 in fp32 above 64 channels), were all as long as the table allows, times the key heads and reads of the cache, below 2^32.
 * Scratch: kda_attn_step_workspace bytes (a function of the sizes, not of the lengths).
 */
typedef struct kda_attn_step_params {
    const void *q;
    void *o;
    float *lse;
    int64_t q_stride;
    int B, T, q_heads;
    float scale;
    int dtype;
    kda_kv_cache cache;
    void *workspace;
    size_t workspace_bytes;
} kda_attn_step_params;

int kda_attn_step(const kda_attn_step_params *p, cudaStream_t stream);
size_t kda_attn_step_workspace(const kda_attn_step_params *p);

#ifdef __cplusplus
}
#endif

#endif /* KDA_ATTENTION_H */
