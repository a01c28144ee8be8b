// Rows of heads (kda_attention.h): the norms of queries and keys with the position rotation, their
// gradient, and the rows' way into the cache and out of it.
//
//   n = x r w, r = (mean x^2 + eps)^(-1/2);  pairs (a, b) of n -> (a cos - b sin, b cos + a sin)
//
// Gradient: g is dy with its pairs turned back, gw = g w, dx = r (gw - x r^2 mean(gw x)), dw = sum g x r.
#include <cuda_fp16.h>

#include "cache_common.cuh"

namespace kda {
namespace {

using namespace mix;

constexpr int kMaxD = 256;
constexpr int kWarps = 8;  // of a block

struct HeadArgs {
    const void *q, *k, *v;      // inputs (backward: also of the forward pass)
    const void *dq_out, *dk_out;
    void *q_out, *k_out;        // outputs (backward: dq, dk)
    const float *qw, *kw;
    const int64_t *freq;
    const int32_t *pos;
    int64_t q_stride, k_stride, v_stride;
    Seqs seqs;
    int Hq, Hk, Hv, D, R;
    bool pairs, cached;         // pairs of neighbours; k and v into the cache
    float eps;
    Cache cache;
    float *partial;             // backward: [blocks][2 D]
    unsigned int *err;
};

// cos and sin of position * freq (2^-64 turns): the 64-bit product is the angle modulo one turn, whatever the position; its
// upper half is rounded to fp32 (off by at most 2^-25 of half a turn).
__device__ __forceinline__ void turn(int64_t freq, int pos, float &c, float &s) {
    const uint64_t t = (uint64_t)freq * (uint64_t)(int64_t)pos;
    sincospif((float)(int32_t)(t >> 32) * 0x1p-31f, &s, &c);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// ---- any width, any alignment: a warp per row, channel lane + 32 j in register j ---------------------
constexpr int kEach = kMaxD / 32;

template <typename T>
__device__ __forceinline__ void any_load(float (&f)[kEach], const void *base, int64_t at, int D, int lane) {
#pragma unroll
    for (int j = 0; j < kEach; ++j) f[j] = lane + 32 * j < D ? to_f(static_cast<const T *>(base)[at + lane + 32 * j]) : 0.f;
}
template <typename T>
__device__ __forceinline__ void any_store(void *base, int64_t at, const float (&f)[kEach], int D, int lane) {
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (lane + 32 * j < D) static_cast<T *>(base)[at + lane + 32 * j] = from_f<T>(f[j]);
}
// Turns the pairs of a row by the angles at `pos` (`sign` -1: back); `mem`: 256 floats of this warp.
__device__ __forceinline__ void any_turn(float (&f)[kEach], float *mem, const HeadArgs &a, int pos, float sign, int lane) {
    if (a.R == 0) return;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kEach; ++j) mem[lane + 32 * j] = f[j];
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int i = lane + 32 * j;
        if (i >= a.R) continue;
        const int half = a.R / 2;
        const bool first = a.pairs ? (i & 1) == 0 : i < half;
        const int other = a.pairs ? i ^ 1 : (first ? i + half : i - half);
        float c, s;
        turn(a.freq[a.pairs ? i >> 1 : (first ? i : i - half)], pos, c, s);
        s *= sign;
        f[j] = first ? f[j] * c - mem[other] * s : f[j] * c + mem[other] * s;
    }
}
// One row into the cache: page < 0 leaves it out.
template <typename T>
__device__ __forceinline__ void any_put(const Cache &c, bool value, const float (&f)[kEach], int page, int head, int slot, int lane) {
    if (page < 0) return;
    const int64_t row = cache_row(c, page, head, slot);
    if (c.ks == nullptr) {
        any_store<T>(value ? c.v : c.k, row * c.D, f, c.D, lane);
        return;
    }
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < kEach; ++j) top = fmaxf(top, finite_abs(f[j]));
    top = warp_max(top);
    bool inf = false;  // an infinity takes the largest exponent, so that it is read back as one
#pragma unroll
    for (int j = 0; j < kEach; ++j) inf |= fabsf(f[j]) == INFINITY;
    const int e = __any_sync(0xffffffffu, inf) ? 120 : row_exponent(top);
    const float unit = pow2(-e);
    uint8_t *to = static_cast<uint8_t *>(value ? c.v : c.k) + row * c.D;
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (lane + 32 * j < c.D) to[lane + 32 * j] = (uint8_t)e4m3_pair(f[j] * unit, 0.f);
    if (lane == 0) (value ? c.vs : c.ks)[cache_scale(c, page, head, slot)] = (uint8_t)(e + 127);
}

// The sequence, position and place of a row.
struct RowAt {
    int pos;         // for the rotation
    int page, slot;  // in the cache; page < 0: not there
};
__device__ __forceinline__ RowAt row_at(const HeadArgs &a, int64_t row, bool places) {
    const SeqAt at = seq_find(a.seqs, row);
    RowAt r;
    r.page = -1;
    r.slot = 0;
    r.pos = (int)(row - at.start);
    if (a.cached) {
        r.pos += cache_len(a.cache, at.s) - (int)(at.end - at.start);
        if (places && r.pos >= 0) r.page = cache_page(a.cache, at.s, r.pos, r.slot);
    }
    if (a.pos != nullptr) r.pos = a.pos[row];
    return r;
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) any_rows_kernel(HeadArgs a) {
    __shared__ float mem[kWarps][kMaxD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x == 0) seq_check(a.seqs, a.err, threadIdx.x, 32 * kWarps);
    const int heads = a.Hq + a.Hk + a.Hv;
    const int64_t items = a.seqs.rows * heads;
    for (int64_t it = (int64_t)blockIdx.x * kWarps + warp; it < items; it += (int64_t)gridDim.x * kWarps) {
        const int64_t row = it / heads;
        const int h = (int)(it - row * heads);
        const bool isq = h < a.Hq, isv = h >= a.Hq + a.Hk;
        const int head = isq ? h : (isv ? h - a.Hq - a.Hk : h - a.Hq);
        const RowAt at = row_at(a, row, !isq);
        float f[kEach];
        const int64_t from = row * (isq ? a.q_stride : isv ? a.v_stride : a.k_stride) + (int64_t)head * a.D;
        any_load<T>(f, isq ? a.q : isv ? a.v : a.k, from, a.D, lane);
        if (!isv) {
            const float *w = isq ? a.qw : a.kw;
            if (w != nullptr) {
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < kEach; ++j) s = fmaf(f[j], f[j], s);
                const float r = rsqrtf(warp_sum(s) / (float)a.D + a.eps);
#pragma unroll
                for (int j = 0; j < kEach; ++j) f[j] = lane + 32 * j < a.D ? f[j] * r * w[lane + 32 * j] : 0.f;
            }
            any_turn(f, mem[warp], a, at.pos, 1.f, lane);
        }
        void *out = isq ? a.q_out : isv ? nullptr : a.k_out;
        if (out != nullptr) any_store<T>(out, (row * (isq ? a.Hq : a.Hk) + head) * a.D, f, a.D, lane);
        if (a.cached && !isq) any_put<T>(a.cache, isv, f, at.page, head, at.slot, lane);
    }
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) any_rows_bwd_kernel(HeadArgs a) {
    __shared__ float mem[kWarps][kMaxD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x == 0) seq_check(a.seqs, a.err, threadIdx.x, 32 * kWarps);
    const int heads = a.Hq + a.Hk;
    const int64_t items = a.seqs.rows * heads;
    float sum[2][kEach] = {};
    for (int64_t it = (int64_t)blockIdx.x * kWarps + warp; it < items; it += (int64_t)gridDim.x * kWarps) {
        const int64_t row = it / heads;
        const int h = (int)(it - row * heads);
        const bool isq = h < a.Hq;
        const int head = isq ? h : h - a.Hq;
        const int64_t dense = (row * (isq ? a.Hq : a.Hk) + head) * a.D;
        float g[kEach], x[kEach];
        any_load<T>(g, isq ? a.dq_out : a.dk_out, dense, a.D, lane);
        any_load<T>(x, isq ? a.q : a.k, row * (isq ? a.q_stride : a.k_stride) + (int64_t)head * a.D, a.D, lane);
        any_turn(g, mem[warp], a, row_at(a, row, false).pos, -1.f, lane);
        const float *w = isq ? a.qw : a.kw;
        if (w != nullptr) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < kEach; ++j) s = fmaf(x[j], x[j], s);
            const float r = rsqrtf(warp_sum(s) / (float)a.D + a.eps);
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                const float gx = g[j] * x[j];
                const float wj = lane + 32 * j < a.D ? w[lane + 32 * j] : 0.f;
                if (isq)
                    sum[0][j] = fmaf(gx, r, sum[0][j]);
                else
                    sum[1][j] = fmaf(gx, r, sum[1][j]);
                m = fmaf(gx, wj, m);
                g[j] *= wj;
            }
            m = warp_sum(m) / (float)a.D * r * r;
#pragma unroll
            for (int j = 0; j < kEach; ++j) g[j] = r * (g[j] - x[j] * m);
        }
        any_store<T>(isq ? a.q_out : a.k_out, dense, g, a.D, lane);
    }
    if (a.partial == nullptr) return;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kEach; ++j) mem[warp][lane + 32 * j] = sum[p][j];
        __syncthreads();
        for (int i = threadIdx.x; i < a.D; i += 32 * kWarps) {
            float t = 0.f;
#pragma unroll
            for (int v = 0; v < kWarps; ++v) t += mem[v][i];
            a.partial[((int64_t)blockIdx.x * 2 + p) * a.D + i] = t;
        }
    }
}

// Rows of the cache into contiguous ones.
template <typename T>
__global__ void __launch_bounds__(32 * kWarps) any_read_kernel(HeadArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x == 0) seq_check(a.seqs, a.err, threadIdx.x, 32 * kWarps);
    const Cache &c = a.cache;
    const int64_t items = a.seqs.rows * 2 * a.Hk;
    for (int64_t it = (int64_t)blockIdx.x * kWarps + warp; it < items; it += (int64_t)gridDim.x * kWarps) {
        const int64_t row = it / (2 * a.Hk);
        const int h = (int)(it - row * 2 * a.Hk);
        const bool isv = h >= a.Hk;
        const int head = isv ? h - a.Hk : h;
        const RowAt at = row_at(a, row, true);
        float f[kEach] = {};
        if (at.page >= 0) {
            const int64_t from = cache_row(c, at.page, head, at.slot);
            const void *base = isv ? c.v : c.k;
            if (c.ks == nullptr) {
                any_load<T>(f, base, from * c.D, c.D, lane);
            } else {
                // a scale of 2^-127 (byte 0), which no row written here has, is below fp32's normal numbers: 0
                const float unit = __uint_as_float((uint32_t)(isv ? c.vs : c.ks)[cache_scale(c, at.page, head, at.slot)] << 23);
#pragma unroll
                for (int j = 0; j < kEach; ++j)
                    if (lane + 32 * j < c.D) {
                        float hi;
                        e4m3_to_f(static_cast<const uint8_t *>(base)[from * c.D + lane + 32 * j], f[j], hi);
                        f[j] *= unit;
                    }
            }
        }
        any_store<T>(isv ? a.q_out : a.k_out, (row * a.Hk + head) * a.D, f, a.D, lane);
    }
}

// ---- host side -------------------------------------------------------------------------------
int elem_size(int dtype) { return dtype == KDA_DTYPE_BF16 ? 2 : 4; }

int sizes_check(int B, int T, const int32_t *cu, int dtype, int heads, int64_t *rows) {
    if (B < 1 || T < 0 || heads < 1) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_F32) return KDA_ERR_UNSUPPORTED;
    *rows = cu != nullptr ? T : (int64_t)B * T;
    if (*rows * heads >= (int64_t)1 << 31) return KDA_ERR_UNSUPPORTED;
    return aligned(cu, 4) ? KDA_OK : KDA_ERR_ALIGNMENT;
}
int stride_check(int64_t given, int64_t dense) { return given != 0 && given < dense ? KDA_ERR_INVALID_ARG : KDA_OK; }

int norm_check(const kda_qk_norm_params &p, bool q_out, bool k_out, int64_t *rows) {
    if (p.q_heads < 1 || p.k_heads < 1 || p.D < 1 || p.R < 0 || p.R % 2 != 0 || p.R > p.D || !(p.eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    const int st = sizes_check(p.B, p.T, p.cu_seqlens, p.dtype, p.q_heads + 2 * p.k_heads, rows);
    if (st != KDA_OK) return st;
    if (p.D > kMaxD) return KDA_ERR_UNSUPPORTED;
    if (stride_check(p.q_stride, (int64_t)p.q_heads * p.D) != KDA_OK || stride_check(p.k_stride, (int64_t)p.k_heads * p.D) != KDA_OK)
        return KDA_ERR_INVALID_ARG;
    if (p.R != 0 && p.freq == nullptr) return KDA_ERR_INVALID_ARG;
    if (*rows != 0 && (p.q == nullptr || p.k == nullptr || (q_out && p.q_out == nullptr) || (k_out && p.k_out == nullptr)))
        return KDA_ERR_INVALID_ARG;
    const size_t e = elem_size(p.dtype);
    if (!aligned(p.q, e) || !aligned(p.k, e) || (q_out && !aligned(p.q_out, e)) || !aligned(p.k_out, e)) return KDA_ERR_ALIGNMENT;
    if (!aligned(p.q_weight, 4) || !aligned(p.k_weight, 4) || !aligned(p.freq, 8) || !aligned(p.positions, 4)) return KDA_ERR_ALIGNMENT;
    // in place: contiguous only, or a row would be written where another one still lies
    if (*rows != 0 && ((q_out && p.q_out == p.q && p.q_stride > (int64_t)p.q_heads * p.D) ||
                       (k_out && p.k_out == p.k && p.k_stride > (int64_t)p.k_heads * p.D)))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

HeadArgs norm_args(const kda_qk_norm_params &p, int64_t rows, unsigned int *err) {
    HeadArgs a{};
    a.q = p.q;
    a.k = p.k;
    a.q_out = p.q_out;
    a.k_out = p.k_out;
    a.qw = p.q_weight;
    a.kw = p.k_weight;
    a.freq = p.freq;
    a.pos = p.positions;
    a.q_stride = p.q_stride != 0 ? p.q_stride : (int64_t)p.q_heads * p.D;
    a.k_stride = p.k_stride != 0 ? p.k_stride : (int64_t)p.k_heads * p.D;
    a.seqs = Seqs{p.cu_seqlens, p.B, p.T, rows};
    a.Hq = p.q_heads;
    a.Hk = p.k_heads;
    a.D = p.D;
    a.R = p.R;
    a.pairs = p.interleaved != 0;
    a.eps = p.eps;
    a.err = err;
    return a;
}

unsigned any_blocks(int64_t items) {
    const int64_t most = (int64_t)sm_count() * 16, need = ceil_div(items, kWarps);
    return (unsigned)(need < most ? need : most);
}

cudaError_t launch_rows(const HeadArgs &a, bool f32, cudaStream_t stream) {
    const unsigned blocks = any_blocks(a.seqs.rows * (a.Hq + a.Hk + a.Hv));
    if (blocks == 0) return cudaErrorInvalidDevice;
    if (f32)
        any_rows_kernel<float><<<blocks, 32 * kWarps, 0, stream>>>(a);
    else
        any_rows_kernel<bf16><<<blocks, 32 * kWarps, 0, stream>>>(a);
    return cudaGetLastError();
}

int bwd_check(const kda_qk_norm_bwd_params &p, int64_t *rows) {
    const int st = norm_check(p.f, false, false, rows);
    if (st != KDA_OK) return st;
    if (*rows != 0 && (p.dq_out == nullptr || p.dk_out == nullptr || p.dq == nullptr || p.dk == nullptr)) return KDA_ERR_INVALID_ARG;
    if ((p.dq_weight != nullptr && p.f.q_weight == nullptr) || (p.dk_weight != nullptr && p.f.k_weight == nullptr))
        return KDA_ERR_INVALID_ARG;
    const size_t e = elem_size(p.f.dtype);
    if (!aligned(p.dq_out, e) || !aligned(p.dk_out, e) || !aligned(p.dq, e) || !aligned(p.dk, e)) return KDA_ERR_ALIGNMENT;
    if (!aligned(p.dq_weight, 4) || !aligned(p.dk_weight, 4)) return KDA_ERR_ALIGNMENT;
    return KDA_OK;
}
unsigned bwd_blocks(const kda_qk_norm_bwd_params &p, int64_t rows) {
    const int64_t most = (int64_t)sm_count() * 4, need = ceil_div(rows * (p.f.q_heads + p.f.k_heads), kWarps);
    return (unsigned)(need < 1 ? 1 : need < most ? need : most);
}
size_t bwd_bytes(const kda_qk_norm_bwd_params &p, int64_t rows) {
    if (p.dq_weight == nullptr && p.dk_weight == nullptr) return 0;
    return (size_t)bwd_blocks(p, rows) * 2 * p.f.D * sizeof(float);
}

}  // namespace
}  // namespace kda

extern "C" {

int kda_qk_norm_fwd(const kda_qk_norm_params *p, cudaStream_t stream) {
    using namespace kda;
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    int64_t rows = 0;
    const int st = norm_check(*p, true, true, &rows);
    if (st != KDA_OK || rows == 0) return st;
    unsigned int *err = nullptr;
    const cudaError_t e = device_error_word(&err);
    if (e != cudaSuccess) return status_of_cuda(e);
    return status_of_cuda(launch_rows(norm_args(*p, rows, err), p->dtype == KDA_DTYPE_F32, stream));
}

int kda_qk_norm_step(const kda_qk_norm_step_params *p, cudaStream_t stream) {
    using namespace kda;
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    int64_t rows = 0;
    int st = norm_check(p->f, true, false, &rows);
    if (st == KDA_OK) st = cache_check(p->cache, p->f.dtype);
    if (st != KDA_OK) return st;
    if (p->cache.heads != p->f.k_heads || p->cache.D != p->f.D || stride_check(p->v_stride, (int64_t)p->f.k_heads * p->f.D) != KDA_OK)
        return KDA_ERR_INVALID_ARG;
    if (rows != 0 && p->v == nullptr) return KDA_ERR_INVALID_ARG;
    if (!aligned(p->v, elem_size(p->f.dtype))) return KDA_ERR_ALIGNMENT;
    if (rows == 0) return KDA_OK;
    unsigned int *err = nullptr;
    const cudaError_t e = device_error_word(&err);
    if (e != cudaSuccess) return status_of_cuda(e);
    HeadArgs a = norm_args(p->f, rows, err);
    a.v = p->v;
    a.v_stride = p->v_stride != 0 ? p->v_stride : (int64_t)p->f.k_heads * p->f.D;
    a.Hv = a.Hk;
    a.cached = true;
    a.cache = cache_args(p->cache, err);
    return status_of_cuda(launch_rows(a, p->f.dtype == KDA_DTYPE_F32, stream));
}

int kda_kv_cache_write(const kda_kv_cache_write_params *p, cudaStream_t stream) {
    using namespace kda;
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    int64_t rows = 0;
    int st = sizes_check(p->B, p->T, p->cu_seqlens, p->dtype, 2 * p->cache.heads, &rows);
    if (st == KDA_OK) st = cache_check(p->cache, p->dtype);
    if (st != KDA_OK) return st;
    const int64_t dense = (int64_t)p->cache.heads * p->cache.D;
    if (stride_check(p->k_stride, dense) != KDA_OK || stride_check(p->v_stride, dense) != KDA_OK) return KDA_ERR_INVALID_ARG;
    if (rows != 0 && (p->k == nullptr || p->v == nullptr)) return KDA_ERR_INVALID_ARG;
    if (!aligned(p->k, elem_size(p->dtype)) || !aligned(p->v, elem_size(p->dtype))) return KDA_ERR_ALIGNMENT;
    if (rows == 0) return KDA_OK;
    unsigned int *err = nullptr;
    const cudaError_t e = device_error_word(&err);
    if (e != cudaSuccess) return status_of_cuda(e);
    HeadArgs a{};
    a.k = p->k;
    a.v = p->v;
    a.k_stride = p->k_stride != 0 ? p->k_stride : dense;
    a.v_stride = p->v_stride != 0 ? p->v_stride : dense;
    a.seqs = Seqs{p->cu_seqlens, p->B, p->T, rows};
    a.Hk = a.Hv = p->cache.heads;
    a.D = p->cache.D;
    a.cached = true;
    a.cache = cache_args(p->cache, err);
    a.err = err;
    return status_of_cuda(launch_rows(a, p->dtype == KDA_DTYPE_F32, stream));
}

int kda_kv_cache_read(const kda_kv_cache_read_params *p, cudaStream_t stream) {
    using namespace kda;
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    int64_t rows = 0;
    int st = sizes_check(p->B, p->T, p->cu_seqlens, p->dtype, 2 * p->cache.heads, &rows);
    if (st == KDA_OK) st = cache_check(p->cache, p->dtype);
    if (st != KDA_OK) return st;
    if (rows != 0 && (p->k == nullptr || p->v == nullptr)) return KDA_ERR_INVALID_ARG;
    if (!aligned(p->k, elem_size(p->dtype)) || !aligned(p->v, elem_size(p->dtype))) return KDA_ERR_ALIGNMENT;
    if (rows == 0) return KDA_OK;
    unsigned int *err = nullptr;
    const cudaError_t e = device_error_word(&err);
    if (e != cudaSuccess) return status_of_cuda(e);
    HeadArgs a{};
    a.k_out = p->k;
    a.q_out = p->v;
    a.seqs = Seqs{p->cu_seqlens, p->B, p->T, rows};
    a.Hk = p->cache.heads;
    a.D = p->cache.D;
    a.cached = true;
    a.cache = cache_args(p->cache, err);
    a.err = err;
    const unsigned blocks = any_blocks(rows * 2 * a.Hk);
    if (blocks == 0) return status_of_cuda(cudaErrorInvalidDevice);
    if (p->dtype == KDA_DTYPE_F32)
        any_read_kernel<float><<<blocks, 32 * kWarps, 0, stream>>>(a);
    else
        any_read_kernel<bf16><<<blocks, 32 * kWarps, 0, stream>>>(a);
    return status_of_cuda(cudaGetLastError());
}

size_t kda_qk_norm_bwd_workspace(const kda_qk_norm_bwd_params *p) {
    using namespace kda;
    int64_t rows = 0;
    if (p == nullptr || bwd_check(*p, &rows) != KDA_OK) return 0;
    return bwd_bytes(*p, rows);
}

int kda_qk_norm_bwd(const kda_qk_norm_bwd_params *p, cudaStream_t stream) {
    using namespace kda;
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    int64_t rows = 0;
    const int st = bwd_check(*p, &rows);
    if (st != KDA_OK) return st;
    const size_t bytes = bwd_bytes(*p, rows);
    if (p->workspace != nullptr && p->workspace_bytes < bytes) return KDA_ERR_INVALID_ARG;
    if (!aligned(p->workspace, 16)) return KDA_ERR_ALIGNMENT;
    if (rows == 0 && bytes == 0) return KDA_OK;
    unsigned int *err = nullptr;
    cudaError_t e = device_error_word(&err);
    if (e != cudaSuccess) return status_of_cuda(e);
    Scratch ws;
    e = ws.get(p->workspace, bytes, stream);
    if (e != cudaSuccess) return status_of_cuda(e);
    HeadArgs a = norm_args(p->f, rows, err);
    a.dq_out = p->dq_out;
    a.dk_out = p->dk_out;
    a.q_out = p->dq;
    a.k_out = p->dk;
    a.partial = static_cast<float *>(ws.ptr);
    const unsigned blocks = bwd_blocks(*p, rows);
    if (p->f.dtype == KDA_DTYPE_F32)
        any_rows_bwd_kernel<float><<<blocks, 32 * kWarps, 0, stream>>>(a);
    else
        any_rows_bwd_kernel<bf16><<<blocks, 32 * kWarps, 0, stream>>>(a);
    e = cudaGetLastError();
    const SumOuts outs{{p->dq_weight, p->dk_weight, nullptr, nullptr}, {p->f.D, p->f.D, 0, 0}};
    if (e == cudaSuccess && bytes != 0) e = launch_sum_partials(a.partial, blocks, 2 * (int64_t)p->f.D, outs, stream);
    return status_of_cuda(ws.release(e));
}

}  // extern "C"
