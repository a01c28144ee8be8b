// RMS norms fused with what stands beside them in a block, and their gradients (kda_mixer.h):
//
//   gated norm   y = x rms(x)^-1 weight act(z)
//   block norm   o = x rms(x)^-1 post_weight;  r' = r + scale act(z) o;  y = r' rms(r')^-1 weight
//
// A row is held in the registers of TPR threads (part of a warp up to 1024 channels, a block
// above), E elements each: every tensor is read and written once, the sums over a row are
// shuffles (and one exchange through shared memory for a block). Bound by memory.
//
// Gradient of n = x i, i = (mean x^2 + eps)^(-1/2), for the gradient g of n:
//   dx = i (g - n mean(g n)).
// The sums over rows (weights, scale) are kept per column in registers while a block goes
// through its rows, added over the block's row groups in a fixed order, and then over the blocks.
#include "mixer_common.cuh"

namespace kda {
namespace {

using namespace mix;

constexpr int kNormMaxD = 8192;

// E elements of a row per thread, as E / V vectors TPR * V apart.
template <int V, int E, int TPR>
struct Cols {
    int lane, D;
    __device__ __forceinline__ int col(int k) const { return (k * TPR + lane) * V; }  // of vector k
    template <typename T>
    __device__ __forceinline__ void load(float (&f)[E], const T *row) const {
#pragma unroll
        for (int k = 0; k < E / V; ++k) {
            const int c = col(k);
            float t[V];
            if (c < D)
                load_vec<T, V>(t, row + c);
            else {
#pragma unroll
                for (int v = 0; v < V; ++v) t[v] = 0.f;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) f[k * V + v] = t[v];
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T *row, const float (&f)[E]) const {
#pragma unroll
        for (int k = 0; k < E / V; ++k) {
            const int c = col(k);
            float t[V];
#pragma unroll
            for (int v = 0; v < V; ++v) t[v] = f[k * V + v];
            if (c < D) store_vec<T, V>(row + c, t);
        }
    }
    // fp32 parameters [D], which need only be 4-byte aligned
    __device__ __forceinline__ void param(float (&f)[E], const float *p) const {
#pragma unroll
        for (int k = 0; k < E / V; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) f[k * V + v] = col(k) < D ? p[col(k) + v] : 0.f;
    }
};

// Sum over the TPR threads of a row; `red` (32 floats per use) serves rows of more than a warp.
template <int TPR>
__device__ __forceinline__ float row_sum(float s, float *red) {
    constexpr int kIn = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int o = kIn / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if constexpr (TPR > 32) {
        __syncthreads();  // red is free again
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
        __syncthreads();
        s = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) s += red[i];
    }
    return s;
}
template <int E>
__device__ __forceinline__ float dot(const float (&a)[E], const float (&b)[E]) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(a[i], b[i], s);
    return s;
}

// Threads of a block: 256, or one row.
template <int TPR>
constexpr int kNormThreads = TPR > 256 ? TPR : 256;

struct NormArgs {
    const void *x, *res, *z, *dy, *dres;
    const float *w, *pw, *scale;
    void *y, *nres, *dx, *dr, *dz;
    float *partial;  // per block: dweight [D], then (block norm) dpost_weight [D], dscale [D]
    int64_t rows;
    int D, silu;
    float eps;
};

template <typename T, int V, int E, int TPR>
__global__ void __launch_bounds__(kNormThreads<TPR>) gated_norm_fwd_kernel(const NormArgs a) {
    constexpr int kRows = kNormThreads<TPR> / TPR;
    __shared__ float red[32];
    const Cols<V, E, TPR> cols{(int)threadIdx.x % TPR, a.D};
    const int64_t stride = (int64_t)gridDim.x * kRows;
    float w[E];
    cols.param(w, a.w);
    // every thread of a warp takes part in the shuffles: rows past the end are read as the last
    for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.rows; base += stride) {
        const int64_t row = base + threadIdx.x / TPR;
        const bool live = row < a.rows;
        const int64_t at = (live ? row : a.rows - 1) * a.D;
        float x[E], z[E];
        cols.load(x, static_cast<const T *>(a.x) + at);
        cols.load(z, static_cast<const T *>(a.z) + at);
        const float inv = rsqrtf(row_sum<TPR>(dot(x, x), red) / a.D + a.eps);
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = x[i] * inv * w[i] * act_value(z[i], a.silu);
        if (live) cols.store(static_cast<T *>(a.y) + at, x);
    }
}

// Adds the row groups' column sums in the order of the groups and writes them for this block.
template <int V, int E, int TPR>
__device__ __forceinline__ void store_column_sums(const Cols<V, E, TPR> &cols, const float (&s)[E], float *out, float *buf) {
    constexpr int kRows = kNormThreads<TPR> / TPR;
    if constexpr (kRows == 1) {
#pragma unroll
        for (int k = 0; k < E / V; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (cols.col(k) < cols.D) out[cols.col(k) + v] = s[k * V + v];
    } else {
        const int group = threadIdx.x / TPR;
        for (int g = 0; g < kRows; ++g) {
            __syncthreads();
            if (g == group)
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    float *at = &buf[i * TPR + cols.lane];
                    *at = g == 0 ? s[i] : *at + s[i];
                }
        }
        __syncthreads();
        if (group == 0)
#pragma unroll
            for (int k = 0; k < E / V; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (cols.col(k) < cols.D) out[cols.col(k) + v] = buf[(k * V + v) * TPR + cols.lane];
        __syncthreads();
    }
}

template <typename T, int V, int E, int TPR>
__global__ void __launch_bounds__(kNormThreads<TPR>) gated_norm_bwd_kernel(const NormArgs a) {
    constexpr int kRows = kNormThreads<TPR> / TPR;
    __shared__ float red[32];
    __shared__ float buf[kRows > 1 ? E * TPR : 1];
    const Cols<V, E, TPR> cols{(int)threadIdx.x % TPR, a.D};
    const int64_t stride = (int64_t)gridDim.x * kRows;
    float w[E], dw[E];
    cols.param(w, a.w);
#pragma unroll
    for (int i = 0; i < E; ++i) dw[i] = 0.f;
    for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.rows; base += stride) {
        const int64_t row = base + threadIdx.x / TPR;
        const bool live = row < a.rows;
        const int64_t at = (live ? row : a.rows - 1) * a.D;
        float x[E], z[E], dy[E];
        cols.load(x, static_cast<const T *>(a.x) + at);
        cols.load(z, static_cast<const T *>(a.z) + at);
        cols.load(dy, static_cast<const T *>(a.dy) + at);
        const float inv = rsqrtf(row_sum<TPR>(dot(x, x), red) / a.D + a.eps);
#pragma unroll
        for (int i = 0; i < E; ++i) {
            float val, der;
            act_both(z[i], a.silu, val, der);
            x[i] *= inv;  // n
            z[i] = dy[i] * x[i] * w[i] * der;
            const float gate = dy[i] * val;
            if (live) dw[i] = fmaf(gate, x[i], dw[i]);
            dy[i] = gate * w[i];  // gradient of n
        }
        if (live) cols.store(static_cast<T *>(a.dz) + at, z);
        const float m = row_sum<TPR>(dot(dy, x), red) / a.D;
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = inv * (dy[i] - x[i] * m);
        if (live) cols.store(static_cast<T *>(a.dx) + at, x);
    }
    store_column_sums(cols, dw, a.partial + (int64_t)blockIdx.x * a.D, buf);
}

// R: the residual's type.
template <typename T, typename R, int V, int E, int TPR>
__global__ void __launch_bounds__(kNormThreads<TPR>) block_norm_fwd_kernel(const NormArgs a) {
    constexpr int kRows = kNormThreads<TPR> / TPR;
    __shared__ float red[32];
    const Cols<V, E, TPR> cols{(int)threadIdx.x % TPR, a.D};
    const int64_t stride = (int64_t)gridDim.x * kRows;
    for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.rows; base += stride) {
        const int64_t row = base + threadIdx.x / TPR;
        const bool live = row < a.rows;
        const int64_t at = (live ? row : a.rows - 1) * a.D;
        float x[E], r[E], t[E];
        cols.load(x, static_cast<const T *>(a.x) + at);
        cols.load(r, static_cast<const R *>(a.res) + at);
        if (a.z != nullptr) cols.load(t, static_cast<const T *>(a.z) + at);
        float inv = 1.f;
        if (a.pw != nullptr) inv = rsqrtf(row_sum<TPR>(dot(x, x), red) / a.D + a.eps);
        if (a.z != nullptr) {
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] *= act_value(t[i], a.silu);
        }
        if (a.pw != nullptr) {
            cols.param(t, a.pw);
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] *= inv * t[i];
        }
        if (a.scale != nullptr) {
            cols.param(t, a.scale);
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] *= t[i];
        }
#pragma unroll
        for (int i = 0; i < E; ++i) r[i] += x[i];
        if (live) cols.store(static_cast<R *>(a.nres) + at, r);
        cols.param(t, a.w);
        const float rinv = rsqrtf(row_sum<TPR>(dot(r, r), red) / a.D + a.eps);
#pragma unroll
        for (int i = 0; i < E; ++i) r[i] *= rinv * t[i];
        if (live) cols.store(static_cast<T *>(a.y) + at, r);
    }
}

template <typename T, typename R, int V, int E, int TPR>
__global__ void __launch_bounds__(kNormThreads<TPR>) block_norm_bwd_kernel(const NormArgs a) {
    constexpr int kRows = kNormThreads<TPR> / TPR;
    __shared__ float red[32];
    __shared__ float buf[kRows > 1 ? E * TPR : 1];
    const Cols<V, E, TPR> cols{(int)threadIdx.x % TPR, a.D};
    const int64_t stride = (int64_t)gridDim.x * kRows;
    float dw[E], dpw[E], dsc[E];
#pragma unroll
    for (int i = 0; i < E; ++i) dw[i] = dpw[i] = dsc[i] = 0.f;
    for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.rows; base += stride) {
        const int64_t row = base + threadIdx.x / TPR;
        const bool live = row < a.rows;
        const int64_t at = (live ? row : a.rows - 1) * a.D;
        float n[E], g[E], t[E], r[E];
        // the forward pass again: n = x / rms (or x), r = r'
        cols.load(n, static_cast<const T *>(a.x) + at);
        cols.load(r, static_cast<const R *>(a.res) + at);
        float inv = 1.f;
        if (a.pw != nullptr) {
            inv = rsqrtf(row_sum<TPR>(dot(n, n), red) / a.D + a.eps);
#pragma unroll
            for (int i = 0; i < E; ++i) n[i] *= inv;
        }
        Raw<T, V> z[E / V];
        if (a.z != nullptr) {
#pragma unroll
            for (int k = 0; k < E / V; ++k) {
                if (cols.col(k) < a.D)
                    z[k].load(static_cast<const T *>(a.z) + at + cols.col(k));
                else
                    z[k].zero();
            }
        }
        // g = scale act(z) post_weight: what multiplies n in r'
#pragma unroll
        for (int k = 0; k < E / V; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int i = k * V + v, c = cols.col(k) + v;
                const bool in = cols.col(k) < a.D;
                float f = 1.f;
                if (a.z != nullptr) f = act_value(z[k].get(v), a.silu);
                if (a.pw != nullptr) f *= in ? a.pw[c] : 0.f;
                if (a.scale != nullptr) f *= in ? a.scale[c] : 0.f;
                g[i] = f;
                r[i] = fmaf(f, n[i], r[i]);
            }
        const float rinv = rsqrtf(row_sum<TPR>(dot(r, r), red) / a.D + a.eps);
        cols.load(t, static_cast<const T *>(a.dy) + at);
#pragma unroll
        for (int k = 0; k < E / V; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int i = k * V + v;
                r[i] *= rinv;
                if (live) dw[i] = fmaf(t[i], r[i], dw[i]);
                t[i] *= cols.col(k) < a.D ? a.w[cols.col(k) + v] : 0.f;
            }
        const float m = row_sum<TPR>(dot(t, r), red) / a.D;
#pragma unroll
        for (int i = 0; i < E; ++i) t[i] = rinv * (t[i] - r[i] * m);
        if (a.dres != nullptr) {
            cols.load(r, static_cast<const R *>(a.dres) + at);
#pragma unroll
            for (int i = 0; i < E; ++i) t[i] += r[i];
        }
        if (live) cols.store(static_cast<R *>(a.dr) + at, t);  // t: gradient of r'
#pragma unroll
        for (int k = 0; k < E / V; ++k) {
            float dz[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int i = k * V + v, c = cols.col(k) + v;
                const bool in = cols.col(k) < a.D;
                const float pw = a.pw != nullptr ? (in ? a.pw[c] : 0.f) : 1.f;
                const float sc = a.scale != nullptr ? (in ? a.scale[c] : 0.f) : 1.f;
                float val = 1.f, der = 0.f;
                if (a.z != nullptr) act_both(z[k].get(v), a.silu, val, der);
                const float tn = t[i] * n[i];
                dz[v] = tn * pw * sc * der;
                if (live) {
                    dsc[i] = fmaf(tn, pw * val, dsc[i]);
                    dpw[i] = fmaf(tn, sc * val, dpw[i]);
                }
                g[i] *= t[i];  // gradient of n
            }
            if (live && a.dz != nullptr && cols.col(k) < a.D) store_vec<T, V>(static_cast<T *>(a.dz) + at + cols.col(k), dz);
        }
        if (a.pw != nullptr) {
            const float mn = row_sum<TPR>(dot(g, n), red) / a.D;
#pragma unroll
            for (int i = 0; i < E; ++i) g[i] = inv * (g[i] - n[i] * mn);
        }
        if (live) cols.store(static_cast<T *>(a.dx) + at, g);
    }
    float *part = a.partial + (int64_t)blockIdx.x * 3 * a.D;
    store_column_sums(cols, dw, part, buf);
    store_column_sums(cols, dpw, part + a.D, buf);
    store_column_sums(cols, dsc, part + 2 * (int64_t)a.D, buf);
}

// ---- host -----------------------------------------------------------------------------------
struct NormPlan {
    int V, E, tpr;
    int64_t blocks;
};

// Threads and elements per row. 8 channels at a time where every row starts on 16 bytes; else
// single channels, in two sizes only.
NormPlan norm_plan(int64_t rows, int D, bool vec, bool block, int per_sm) {
    NormPlan q{};
    q.V = vec ? 8 : 1;
    if (!vec) {
        q.tpr = D <= 1024 ? 32 : 512;
        q.E = D <= 1024 ? 32 : 16;
    } else if (block) {  // up to six tensors of a row in registers: at most 16 elements each
        if (D <= 256)
            q.tpr = 32, q.E = 8;
        else if (D <= 2048)
            q.tpr = 256, q.E = 8;
        else
            q.tpr = D <= 4096 ? 256 : 512, q.E = 16;
    } else {
        if (D <= 64)
            q.tpr = 8, q.E = 8;
        else if (D <= 128)
            q.tpr = 16, q.E = 8;
        else if (D <= 256)
            q.tpr = 32, q.E = 8;
        else if (D <= 1024)
            q.tpr = 32, q.E = 32;
        else if (D <= 2048)
            q.tpr = 256, q.E = 8;
        else
            q.tpr = D <= 4096 ? 256 : 512, q.E = 16;
    }
    const int per_block = q.tpr > 256 ? 1 : 256 / q.tpr;
    const int64_t most = (int64_t)per_sm * (sm_count() > 0 ? sm_count() : 1);
    q.blocks = ceil_div(rows, per_block);
    if (q.blocks > most) q.blocks = most;
    if (q.blocks < 1) q.blocks = 1;
    return q;
}

#define KDA_NORM_LAUNCH(kernel, V_, E_, TPR_, ...) \
    if (q.V == V_ && q.E == E_ && q.tpr == TPR_) { \
        kernel<__VA_ARGS__, V_, E_, TPR_><<<(unsigned)q.blocks, kNormThreads<TPR_>, 0, stream>>>(a); \
        return cudaGetLastError(); \
    }
#define KDA_NORM_BLOCK_SIZES(kernel, ...) \
    KDA_NORM_LAUNCH(kernel, 8, 8, 32, __VA_ARGS__) \
    KDA_NORM_LAUNCH(kernel, 8, 8, 256, __VA_ARGS__) \
    KDA_NORM_LAUNCH(kernel, 8, 16, 256, __VA_ARGS__) \
    KDA_NORM_LAUNCH(kernel, 8, 16, 512, __VA_ARGS__) \
    KDA_NORM_LAUNCH(kernel, 1, 32, 32, __VA_ARGS__) \
    KDA_NORM_LAUNCH(kernel, 1, 16, 512, __VA_ARGS__)
#define KDA_NORM_GATED_SIZES(kernel, ...) \
    KDA_NORM_BLOCK_SIZES(kernel, __VA_ARGS__) \
    KDA_NORM_LAUNCH(kernel, 8, 8, 8, __VA_ARGS__) \
    KDA_NORM_LAUNCH(kernel, 8, 8, 16, __VA_ARGS__) \
    KDA_NORM_LAUNCH(kernel, 8, 32, 32, __VA_ARGS__)

template <typename T>
cudaError_t launch_gated(const NormPlan &q, const NormArgs &a, bool bwd, cudaStream_t stream) {
    if (bwd) {
        KDA_NORM_GATED_SIZES(gated_norm_bwd_kernel, T)
    } else {
        KDA_NORM_GATED_SIZES(gated_norm_fwd_kernel, T)
    }
    return cudaErrorInvalidValue;
}
template <typename T, typename R>
cudaError_t launch_block(const NormPlan &q, const NormArgs &a, bool bwd, cudaStream_t stream) {
    if (bwd) {
        KDA_NORM_BLOCK_SIZES(block_norm_bwd_kernel, T, R)
    } else {
        KDA_NORM_BLOCK_SIZES(block_norm_fwd_kernel, T, R)
    }
    return cudaErrorInvalidValue;
}

int elem_size(int dtype) { return dtype == KDA_DTYPE_BF16 ? 2 : 4; }

bool vec_ok(int D, const void *const *ptrs, int n) {
    bool ok = D % 8 == 0;
    for (int i = 0; i < n; ++i) ok = ok && aligned(ptrs[i], 16);
    return ok;
}
int aligned_status(const void *const *ptrs, int n, size_t bytes) {
    for (int i = 0; i < n; ++i)
        if (!aligned(ptrs[i], bytes)) return KDA_ERR_ALIGNMENT;
    return KDA_OK;
}

int size_check(int64_t rows, int D, float eps, int dtype) {
    if (rows < 0 || D < 1 || !(eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_F32) return KDA_ERR_UNSUPPORTED;
    if (D > kNormMaxD) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

int gated_check(const kda_gated_norm_params &p, bool fwd) {
    const int st = size_check(p.rows, p.D, p.eps, p.dtype);
    if (st != KDA_OK) return st;
    if (p.activation != KDA_ACT_SILU && p.activation != KDA_ACT_SIGMOID) return KDA_ERR_UNSUPPORTED;
    if (p.weight == nullptr || (p.rows != 0 && (p.x == nullptr || p.z == nullptr || (fwd && p.y == nullptr))))
        return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {p.x, p.z, fwd ? p.y : nullptr};
    if (!aligned(p.weight, 4)) return KDA_ERR_ALIGNMENT;
    return aligned_status(ptrs, 3, elem_size(p.dtype));
}

NormArgs gated_args(const kda_gated_norm_params &p) {
    NormArgs a{};
    a.x = p.x;
    a.z = p.z;
    a.w = p.weight;
    a.y = p.y;
    a.rows = p.rows;
    a.D = p.D;
    a.silu = p.activation == KDA_ACT_SILU;
    a.eps = p.eps;
    return a;
}

int gated_bwd_check(const kda_gated_norm_bwd_params &p) {
    const int st = gated_check(p.f, false);
    if (st != KDA_OK) return st;
    if (p.dweight == nullptr || (p.f.rows != 0 && (p.dy == nullptr || p.dx == nullptr || p.dz == nullptr)))
        return KDA_ERR_INVALID_ARG;
    const void *ptrs[] = {p.dy, p.dx, p.dz};
    if (!aligned(p.dweight, 4)) return KDA_ERR_ALIGNMENT;
    return aligned_status(ptrs, 3, elem_size(p.f.dtype));
}
NormPlan gated_bwd_plan(const kda_gated_norm_bwd_params &p) {
    const void *ptrs[] = {p.f.x, p.f.z, p.dy, p.dx, p.dz};
    return norm_plan(p.f.rows, p.f.D, vec_ok(p.f.D, ptrs, 5), false, 4);
}

int block_check(const kda_block_norm_params &p, bool fwd) {
    const int st = size_check(p.rows, p.D, p.eps, p.dtype);
    if (st != KDA_OK) return st;
    if (p.res_dtype != KDA_DTYPE_F32 && p.res_dtype != p.dtype) return KDA_ERR_UNSUPPORTED;
    if (p.z != nullptr && p.activation != KDA_ACT_SILU && p.activation != KDA_ACT_SIGMOID) return KDA_ERR_UNSUPPORTED;
    if (p.weight == nullptr) return KDA_ERR_INVALID_ARG;
    if (p.rows != 0 && (p.x == nullptr || p.residual == nullptr || (fwd && (p.y == nullptr || p.new_residual == nullptr))))
        return KDA_ERR_INVALID_ARG;
    const void *f32[] = {p.weight, p.post_weight, p.scale};
    const void *ptrs[] = {p.x, p.z, fwd ? p.y : nullptr};
    const void *res[] = {p.residual, fwd ? p.new_residual : nullptr};
    if (aligned_status(f32, 3, 4) != KDA_OK || aligned_status(res, 2, elem_size(p.res_dtype)) != KDA_OK) return KDA_ERR_ALIGNMENT;
    return aligned_status(ptrs, 3, elem_size(p.dtype));
}

NormArgs block_args(const kda_block_norm_params &p) {
    NormArgs a{};
    a.x = p.x;
    a.res = p.residual;
    a.w = p.weight;
    a.pw = p.post_weight;
    a.z = p.z;
    a.scale = p.scale;
    a.y = p.y;
    a.nres = p.new_residual;
    a.rows = p.rows;
    a.D = p.D;
    a.silu = p.activation == KDA_ACT_SILU;
    a.eps = p.eps;
    return a;
}

int block_bwd_check(const kda_block_norm_bwd_params &p) {
    const int st = block_check(p.f, false);
    if (st != KDA_OK) return st;
    if (p.dweight == nullptr || (p.f.rows != 0 && (p.dy == nullptr || p.dx == nullptr || p.dresidual == nullptr)))
        return KDA_ERR_INVALID_ARG;
    if ((p.dz != nullptr && p.f.z == nullptr) || (p.dpost_weight != nullptr && p.f.post_weight == nullptr) ||
        (p.dscale != nullptr && p.f.scale == nullptr))
        return KDA_ERR_INVALID_ARG;
    const void *f32[] = {p.dweight, p.dpost_weight, p.dscale};
    const void *ptrs[] = {p.dy, p.dx, p.dz};
    const void *res[] = {p.dres, p.dresidual};
    if (aligned_status(f32, 3, 4) != KDA_OK || aligned_status(res, 2, elem_size(p.f.res_dtype)) != KDA_OK) return KDA_ERR_ALIGNMENT;
    return aligned_status(ptrs, 3, elem_size(p.f.dtype));
}
NormPlan block_bwd_plan(const kda_block_norm_bwd_params &p) {
    const void *ptrs[] = {p.f.x, p.f.z, p.f.residual, p.dy, p.dres, p.dx, p.dresidual, p.dz};
    return norm_plan(p.f.rows, p.f.D, vec_ok(p.f.D, ptrs, 8), true, 2);
}

cudaError_t run_block(const kda_block_norm_params &p, const NormPlan &q, const NormArgs &a, bool bwd, cudaStream_t stream) {
    if (p.dtype == KDA_DTYPE_F32) return launch_block<float, float>(q, a, bwd, stream);
    if (p.res_dtype == KDA_DTYPE_F32) return launch_block<bf16, float>(q, a, bwd, stream);
    return launch_block<bf16, bf16>(q, a, bwd, stream);
}

}  // namespace
}  // namespace kda

extern "C" {

int kda_gated_norm_fwd(const kda_gated_norm_params *p, cudaStream_t stream) {
    using namespace kda;
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    const int st = gated_check(*p, true);
    if (st != KDA_OK || p->rows == 0) return st;
    const void *ptrs[] = {p->x, p->z, p->y};
    const NormPlan q = norm_plan(p->rows, p->D, vec_ok(p->D, ptrs, 3), false, 16);
    const NormArgs a = gated_args(*p);
    return status_of_cuda(p->dtype == KDA_DTYPE_F32 ? launch_gated<float>(q, a, false, stream)
                                                    : launch_gated<bf16>(q, a, false, stream));
}

size_t kda_gated_norm_bwd_workspace(const kda_gated_norm_bwd_params *p) {
    using namespace kda;
    if (p == nullptr || gated_bwd_check(*p) != KDA_OK) return 0;
    return (size_t)gated_bwd_plan(*p).blocks * p->f.D * sizeof(float);
}

int kda_gated_norm_bwd(const kda_gated_norm_bwd_params *p, cudaStream_t stream) {
    using namespace kda;
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    const int st = gated_bwd_check(*p);
    if (st != KDA_OK) return st;
    const NormPlan q = gated_bwd_plan(*p);
    const size_t bytes = (size_t)q.blocks * p->f.D * sizeof(float);
    if (p->workspace != nullptr && p->workspace_bytes < bytes) return KDA_ERR_INVALID_ARG;
    if (!aligned(p->workspace, 16)) return KDA_ERR_ALIGNMENT;
    NormArgs a = gated_args(p->f);
    a.dy = p->dy;
    a.dx = p->dx;
    a.dz = p->dz;
    Scratch ws;
    cudaError_t e = ws.get(p->workspace, bytes, stream);
    if (e != cudaSuccess) return status_of_cuda(e);
    a.partial = static_cast<float *>(ws.ptr);
    e = p->f.dtype == KDA_DTYPE_F32 ? launch_gated<float>(q, a, true, stream) : launch_gated<bf16>(q, a, true, stream);
    const SumOuts outs{{p->dweight, nullptr, nullptr, nullptr}, {p->f.D, 0, 0, 0}};
    if (e == cudaSuccess) e = launch_sum_partials(a.partial, q.blocks, p->f.D, outs, stream);
    return status_of_cuda(ws.release(e));
}

int kda_block_norm_fwd(const kda_block_norm_params *p, cudaStream_t stream) {
    using namespace kda;
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    const int st = block_check(*p, true);
    if (st != KDA_OK || p->rows == 0) return st;
    const void *ptrs[] = {p->x, p->z, p->residual, p->y, p->new_residual};
    const NormPlan q = norm_plan(p->rows, p->D, vec_ok(p->D, ptrs, 5), true, 16);
    return status_of_cuda(run_block(*p, q, block_args(*p), false, stream));
}

size_t kda_block_norm_bwd_workspace(const kda_block_norm_bwd_params *p) {
    using namespace kda;
    if (p == nullptr || block_bwd_check(*p) != KDA_OK) return 0;
    return (size_t)block_bwd_plan(*p).blocks * 3 * p->f.D * sizeof(float);
}

int kda_block_norm_bwd(const kda_block_norm_bwd_params *p, cudaStream_t stream) {
    using namespace kda;
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    const int st = block_bwd_check(*p);
    if (st != KDA_OK) return st;
    const NormPlan q = block_bwd_plan(*p);
    const size_t bytes = (size_t)q.blocks * 3 * p->f.D * sizeof(float);
    if (p->workspace != nullptr && p->workspace_bytes < bytes) return KDA_ERR_INVALID_ARG;
    if (!aligned(p->workspace, 16)) return KDA_ERR_ALIGNMENT;
    NormArgs a = block_args(p->f);
    a.dy = p->dy;
    a.dres = p->dres;
    a.dx = p->dx;
    a.dr = p->dresidual;
    a.dz = p->dz;
    Scratch ws;
    cudaError_t e = ws.get(p->workspace, bytes, stream);
    if (e != cudaSuccess) return status_of_cuda(e);
    a.partial = static_cast<float *>(ws.ptr);
    e = run_block(p->f, q, a, true, stream);
    const SumOuts outs{{p->dweight, p->dpost_weight, p->dscale, nullptr}, {p->f.D, p->f.D, p->f.D, 0}};
    if (e == cudaSuccess) e = launch_sum_partials(a.partial, q.blocks, 3 * (int64_t)p->f.D, outs, stream);
    return status_of_cuda(ws.release(e));
}

}  // extern "C"
