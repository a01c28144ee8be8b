/*
 * kda_mixer.h — C ABI of the token-mixer operators that stand around the recurrences of
 * kda.h in a model's block, for NVIDIA GB300 (sm_103a), in the same library:
 *
 *   kda_conv_*        the short causal depthwise convolution before the recurrence
 *   kda_scan_*        the selective state space scan: a recurrence with one decay per
 *                     (token, channel, state), which kda_chunk_fwd cannot express (its gate
 *                     is shared by the d_v channels of a head)
 *   kda_gated_norm_*  the RMS norm of the recurrence's output, times a gate
 *   kda_block_norm_*  the residual update at the end of a block (norm, gate and scale of the
 *                     block's output) and the norm before the next block
 *
 * each with its backward pass; the convolution and the scan also with a form for single
 * tokens that updates the sequences' states in place.
 *
 * Common to all calls, as in kda.h: tensor pointers are DEVICE pointers of the current device; data tensors are
 * bf16 or fp32 (`dtype`, KDA_DTYPE_*), parameters and recurrence states fp32; sums, states and
 * norms are held in fp32 and a result is rounded to its tensor's type once. Calls are
 * asynchronous on `stream`, thread-safe, and fully overwrite their outputs, which must not
 * alias an input unless stated; the same inputs give bitwise equal outputs (no
 * atomics on outputs). Packed sequences: cu_seqlens != NULL holds B + 1 device int32 offsets
 * of B sequences in T rows; a malformed array (offsets that decrease, cu_seqlens[0] != 0 or
 * cu_seqlens[B] != T) leaves the outputs undefined, touches no memory outside
 * the tensors, and raises KDA_DEVICE_ERR_SEQLENS (kda_get_device_error). Empty sequences and
 * T == 0 are valid.
 *
 * Token strides: the convolution's x and the scan's u, dt, B, C and z may be slices of wider
 * tensors. Their `*_stride` is the distance in elements between consecutive tokens (all B x T tokens
 * evenly spaced, the channels of a token contiguous); 0 means contiguous. Outputs and all other
 * tensors, the norms' x and z among them, are contiguous. Pointers are aligned to their element
 * type; where all rows are aligned for it several elements are read at a time, otherwise one.
 *
 * Scratch: the calls that need it say so; it is `workspace` (16-byte aligned, at least the
 * bytes that the matching *_workspace function returns, free for reuse when the call's work on
 * `stream` has ended) or, with workspace == NULL, stream-ordered memory of the
 * library's pool, freed on the same stream.
 *
 * Errors: as in kda.h; nothing is launched when a status other than KDA_OK or KDA_ERR_CUDA is
 * returned.
 */
#ifndef KDA_MIXER_H
#define KDA_MIXER_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_ACT_NONE 0
#define KDA_ACT_SILU 1    /* x / (1 + e^-x) */
#define KDA_ACT_SIGMOID 2 /* 1 / (1 + e^-x) */

/*
 * kda_conv_fwd — short causal depthwise convolution over the tokens of each sequence:
 *
 *     y_t[c] = act(bias[c] + sum_{j < W} weight[c][j] x_{t - (W - 1) + j}[c])
 *
 * where x at the W - 1 tokens before the sequence is the initial state s0, or zero.
 *   x, y      [B, T, D] (or [1, T, D] packed), `dtype`; x with token stride x_stride
 *   weight    [D, W] fp32, W in {2, 3, 4};  bias [D] fp32 or NULL
 *   s0, st    [N, W - 1, D] `dtype`, the W - 1 inputs before the first token and up to the last
 *             one, oldest first, N the number of sequences; either may be NULL (s0: zeros);
 *             st must not be s0 (KDA_ERR_INVALID_ARG; kda_conv_step updates in place)
 *   activation KDA_ACT_NONE or KDA_ACT_SILU
 */
typedef struct kda_conv_params {
    const void *x;
    const float *weight, *bias;
    const void *s0;
    void *y, *st;
    int64_t x_stride;
    int B, T, D, W;
    const int32_t *cu_seqlens;
    int dtype, activation;
} kda_conv_params;

int kda_conv_fwd(const kda_conv_params *p, cudaStream_t stream);

/* kda_conv_step — the same for the next T tokens (typically one) of each of B sequences, each
 * walked by itself: st may be s0, the states are then updated in place. cu_seqlens must be
 * NULL, s0 and st are required. */
int kda_conv_step(const kda_conv_params *p, cudaStream_t stream);

/*
 * kda_conv_bwd — gradients of sum(dy * y) + sum(dst * st) with respect to x, weight, bias and
 * s0. dst NULL: no gradient reaches the final states; ds0, dbias NULL: not wanted (s0 may be
 * NULL with ds0 given: the gradient at zero states). Scratch: kda_conv_bwd_workspace bytes.
 *   dy, dx [B, T, D], dst, ds0 [N, W - 1, D] `dtype`; dweight [D, W], dbias [D] fp32
 */
typedef struct kda_conv_bwd_params {
    const void *x;
    const float *weight, *bias;
    const void *s0, *dy, *dst;
    void *dx;
    float *dweight, *dbias;
    void *ds0;
    int64_t x_stride;
    int B, T, D, W;
    const int32_t *cu_seqlens;
    int dtype, activation;
    void *workspace;
    size_t workspace_bytes;
} kda_conv_bwd_params;

int kda_conv_bwd(const kda_conv_bwd_params *p, cudaStream_t stream);
size_t kda_conv_bwd_workspace(const kda_conv_bwd_params *p);

/*
 * kda_scan_fwd — selective state space scan. For each sequence and channel d, with N states:
 *
 *     s_t    = dt_t[d] + dt_bias[d];  delta_t = softplus(s_t) with dt_softplus, else s_t
 *     h_t[n] = exp(delta_t A[d][n]) h_{t-1}[n] + delta_t u_t[d] B_t[g][n]
 *     y_t[d] = (sum_n C_t[g][n] h_t[n] + D[d] u_t[d]) * silu(z_t[d])
 *
 * with g = d / (channels / G), D and z each optional (NULL: no skip, no gate).
 *   u, dt, z, y  [B, T, channels] `dtype`;  B, C [B, T, G, N] `dtype`
 *   A [channels, N], D, dt_bias [channels] fp32 (dt_bias may be NULL)
 *   h0, ht       [N_seq, channels, N] fp32, either may be NULL (h0: zeros); ht must not be h0
 *                (KDA_ERR_INVALID_ARG; kda_scan_step updates in place)
 * 1 <= N <= 64; channels divisible by G; channels N and the number of tokens below 2^31.
 * Where one pass over the tokens would leave most of the GPU idle (few channels and sequences)
 * the tokens are cut into pieces: scratch of kda_scan_fwd_workspace bytes.
 */
typedef struct kda_scan_params {
    const void *u, *dt;
    const float *A;
    const void *B, *C;
    const float *D;
    const void *z;
    const float *dt_bias, *h0;
    void *y;
    float *ht;
    int64_t u_stride, dt_stride, B_stride, C_stride, z_stride;
    int batch, T, channels, N, G;
    const int32_t *cu_seqlens;
    int dtype, dt_softplus;
    void *workspace;
    size_t workspace_bytes;
} kda_scan_params;

int kda_scan_fwd(const kda_scan_params *p, cudaStream_t stream);
size_t kda_scan_fwd_workspace(const kda_scan_params *p);

/* kda_scan_step — the same for the next T tokens (typically one) of each of `batch` sequences:
 * ht may be h0, the states are then updated in place. cu_seqlens must be NULL, h0 and ht are
 * required, no scratch. */
int kda_scan_step(const kda_scan_params *p, cudaStream_t stream);

/*
 * kda_scan_bwd — gradients of sum(dy * y) + sum(dht * ht) for the forward pass `f` (its y, ht
 * and workspace are not read). The states are recomputed from the inputs. dht NULL: no
 * gradient reaches the final states; dD, dz, ddt_bias, dh0 NULL: not wanted (dD must be NULL
 * without D, dz without z).
 *   du, ddt, dz like u (contiguous); dB, dC like B (contiguous; sums over the channels of a
 *   group); dA [channels, N], dD, ddt_bias [channels], dh0 like h0: fp32
 * ddt is the gradient with respect to dt as given (before bias and softplus). Scratch:
 * kda_scan_bwd_workspace bytes, all fp32: per token channels (N + 1) / 4 bytes of states and step sizes (at
 * every 16th token; channels (N + 1) / 2, at every 8th, for N > 32) and 8 N bytes for every block of 64
 * channels (shares of dB and dC; a group's last block may be smaller); per chunk 12 channels (N + 1) bytes of
 * what the chunks hand over. Chunks have 32 tokens or, where so many are not needed to fill the GPU, more.
 */
typedef struct kda_scan_bwd_params {
    kda_scan_params f;
    const void *dy;
    const float *dht;
    void *du, *ddt;
    float *dA;
    void *dB, *dC;
    float *dD;
    void *dz;
    float *ddt_bias, *dh0;
    void *workspace;
    size_t workspace_bytes;
} kda_scan_bwd_params;

int kda_scan_bwd(const kda_scan_bwd_params *p, cudaStream_t stream);
size_t kda_scan_bwd_workspace(const kda_scan_bwd_params *p);

/*
 * kda_gated_norm_fwd — per row (a token's head) of D channels:
 *
 *     y = x / sqrt(mean(x^2) + eps) * weight * act(z)
 *
 *   x, z, y [rows, D] `dtype`, weight [D] fp32; activation KDA_ACT_SILU or KDA_ACT_SIGMOID;
 *   1 <= D <= 8192
 */
typedef struct kda_gated_norm_params {
    const void *x, *z;
    const float *weight;
    void *y;
    int64_t rows;
    int D;
    float eps;
    int dtype, activation;
} kda_gated_norm_params;

int kda_gated_norm_fwd(const kda_gated_norm_params *p, cudaStream_t stream);

/* kda_gated_norm_bwd — dx, dz (like x) and dweight [D] fp32 for the gradient dy of y (the y of
 * `f` is not read). Scratch: kda_gated_norm_bwd_workspace bytes. */
typedef struct kda_gated_norm_bwd_params {
    kda_gated_norm_params f;
    const void *dy;
    void *dx, *dz;
    float *dweight;
    void *workspace;
    size_t workspace_bytes;
} kda_gated_norm_bwd_params;

int kda_gated_norm_bwd(const kda_gated_norm_bwd_params *p, cudaStream_t stream);
size_t kda_gated_norm_bwd_workspace(const kda_gated_norm_bwd_params *p);

/*
 * kda_block_norm_fwd — the end of a block and the start of the next, per row of D channels:
 *
 *     o  = x / sqrt(mean(x^2) + eps) * post_weight     (o = x without post_weight)
 *     r' = residual + scale * act(z) * o               (no gate without z, scale 1 without scale)
 *     y  = r' / sqrt(mean(r'^2) + eps) * weight
 *
 *   x (the block's output), z, y [rows, D] `dtype`; residual, new_residual (r') [rows, D]
 *   `res_dtype`: `dtype` or KDA_DTYPE_F32; weight, post_weight, scale [D] fp32.
 *   new_residual may be residual (updated in place). 1 <= D <= 8192. The norm of r' is taken
 *   before r' is rounded to res_dtype.
 */
typedef struct kda_block_norm_params {
    const void *x, *residual;
    const float *weight, *post_weight;
    const void *z;
    const float *scale;
    void *y, *new_residual;
    int64_t rows;
    int D;
    float eps;
    int dtype, res_dtype, activation;
} kda_block_norm_params;

int kda_block_norm_fwd(const kda_block_norm_params *p, cudaStream_t stream);

/* kda_block_norm_bwd — for the gradients dy of y and dres of r' (dres NULL: none), the
 * gradients dx, dz (like x), dresidual (like residual; may be dres) and dweight, dpost_weight,
 * dscale [D] fp32; dz, dpost_weight and dscale must be NULL where the forward pass has no
 * such argument and may be NULL where it has (not wanted). The y and new_residual of `f` are
 * not read; residual is the tensor before the update. Scratch: kda_block_norm_bwd_workspace
 * bytes. */
typedef struct kda_block_norm_bwd_params {
    kda_block_norm_params f;
    const void *dy, *dres;
    void *dx, *dresidual;
    float *dweight, *dpost_weight;
    void *dz;
    float *dscale;
    void *workspace;
    size_t workspace_bytes;
} kda_block_norm_bwd_params;

int kda_block_norm_bwd(const kda_block_norm_bwd_params *p, cudaStream_t stream);
size_t kda_block_norm_bwd_workspace(const kda_block_norm_bwd_params *p);

#ifdef __cplusplus
}
#endif

#endif /* KDA_MIXER_H */
