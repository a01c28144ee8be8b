// RMS norms fused with what stands beside them in a block, and their gradients (kda_mixer.h):
//
//   gated norm   y = x rms(x)^-1 weight act(z)
//   block norm   o = x rms(x)^-1 post_weight;  r' = r + scale act(z) o;  y = r' rms(r')^-1 weight
//
// A row is held in the registers of TPR threads, 8 (above 4096 channels 16) elements each: every tensor is
// read and written once. Sums over a row are shuffles, above 256 channels with one exchange through
// shared memory and one barrier each. The next row's loads are issued before the current row is
// worked on. Bound by memory: 16384 x 4096 block norm (bf16, fp32 residual) 144 us, 6.5 TB/s, its gradient on 8192
// rows 140 us, 5.3 TB/s; 524288 x 128 gated norm 68 us, 5.9 TB/s, its gradient on half the rows 64 us, 5.3 TB/s.
//
// Gradient of n = x i, i = (mean x^2 + eps)^(-1/2), for the gradient g of n:
//   dx = i (g - n mean(g n)) = i (g - x i^2 mean(g x)),
// so that the sum of g x can go with another one, before i is known.
// The sums over rows (weights, scale) are kept per column (registers; shared memory for 16 elements per
// thread) while a block goes through its rows, added over the block's row groups in a fixed order,
// and then over the blocks.
#include "mixer_common.cuh"

namespace kda {
namespace {

using namespace mix;

constexpr int kNormMaxD = 8192;

// E elements of a row per thread, as E / V vectors TPR * V apart.
template <int V, int E, int TPR>
struct Cols {
    static constexpr int K = E / V;
    int lane, D;
    __device__ __forceinline__ int col(int k) const { return (k * TPR + lane) * V; }  // of vector k
    __device__ __forceinline__ bool in(int k) const { return col(k) < D; }
    template <typename T>
    __device__ __forceinline__ void fetch(Raw<T, V> (&r)[K], const void *base, int64_t at) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (in(k))
                r[k].load(static_cast<const T *>(base) + at + col(k));
            else
                r[k].zero();
        }
    }
    template <typename T>
    __device__ __forceinline__ void unpack(float (&f)[E], const Raw<T, V> (&r)[K]) const {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) f[k * V + v] = r[k].get(v);
    }
    template <typename T>
    __device__ __forceinline__ void store(void *base, int64_t at, const float (&f)[E]) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float t[V];
#pragma unroll
            for (int v = 0; v < V; ++v) t[v] = f[k * V + v];
            if (in(k)) store_vec<T, V>(static_cast<T *>(base) + at + col(k), t);
        }
    }
    // from a row of shared memory that this thread filled itself
    __device__ __forceinline__ void own(float (&f)[E], const float *mem) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float t[V];
            load_vec<float, V>(t, mem + (k * TPR + lane) * V);
#pragma unroll
            for (int v = 0; v < V; ++v) f[k * V + v] = t[v];
        }
    }
    __device__ __forceinline__ void keep(float *mem, const float (&f)[E]) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float t[V];
#pragma unroll
            for (int v = 0; v < V; ++v) t[v] = f[k * V + v];
            store_vec<float, V>(mem + (k * TPR + lane) * V, t);
        }
    }
    // fp32 parameters [D]; f = 1 without them
    __device__ __forceinline__ void param(float (&f)[E], const float *p) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float t[V];
#pragma unroll
            for (int v = 0; v < V; ++v) t[v] = 1.f;
            if (p != nullptr && in(k)) load_vec<float, V>(t, p + col(k));
#pragma unroll
            for (int v = 0; v < V; ++v) f[k * V + v] = t[v];
        }
    }
};

// Sums of one or two values over the TPR threads of a row. Rows of more than a warp exchange through
// `red` (two buffers of 32 pairs, used in turn: one barrier per sum is enough).
template <int TPR>
struct RowSum {
    float2 *red;
    int turn = 0;
    template <int M>
    __device__ __forceinline__ void run(float (&v)[M]) {
        constexpr int kIn = TPR < 32 ? TPR : 32;
#pragma unroll
        for (int o = kIn / 2; o > 0; o >>= 1)
#pragma unroll
            for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
        if constexpr (TPR > 32) {
            float *buf = reinterpret_cast<float *>(red + 32 * turn);
            turn ^= 1;
            const int warp = threadIdx.x >> 5;
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int m = 0; m < M; ++m) buf[warp * M + m] = v[m];
            __syncthreads();
            // lane l takes warp l % kWarps of this row, then the warps' sums are added across lanes
            constexpr int kWarps = TPR / 32;
            const int first = warp / kWarps * kWarps, lane = threadIdx.x & (kWarps - 1);
#pragma unroll
            for (int m = 0; m < M; ++m) v[m] = buf[(first + lane) * M + m];
#pragma unroll
            for (int o = kWarps / 2; o > 0; o >>= 1)
#pragma unroll
                for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
        }
    }
    __device__ __forceinline__ float operator()(float a) {
        float v[1] = {a};
        run(v);
        return v[0];
    }
    __device__ __forceinline__ float2 operator()(float a, float b) {
        float v[2] = {a, b};
        run(v);
        return make_float2(v[0], v[1]);
    }
};

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
template <int TPR>
constexpr int kNormRows = kNormThreads<TPR> / TPR;

struct NormArgs {
    const void *x, *res, *z, *dy, *dres;
    const float *w, *pw, *scale;
    void *y, *nres, *dx, *dr, *dz;
    float *partial;  // per block: dweight [D], then (block norm) dpost_weight [D], dscale [D]
    int64_t rows;
    int D, silu;
    float eps;
};

// Calls row(at, live) for this thread's rows, at = the row's first element: fetch(at) has been
// issued for it before the previous row was worked on. Every thread of a block takes part in every
// turn (the sums need them): rows past the end are the last row again, not live.
// before() comes between the first row's fetch and its turn.
template <int TPR, typename F, typename P, typename B>
__device__ __forceinline__ void for_rows(const NormArgs &a, F fetch, P before, B body) {
    const int64_t step = (int64_t)gridDim.x * kNormRows<TPR>;
    int64_t base = (int64_t)blockIdx.x * kNormRows<TPR>;
    if (base >= a.rows) return;
    auto place = [&](int64_t b) {
        const int64_t r = b + threadIdx.x / TPR;
        return (r < a.rows ? r : a.rows - 1) * a.D;
    };
    fetch(place(base));
    before();
    for (; base < a.rows; base += step) body(place(base), base + threadIdx.x / TPR < a.rows, base + step < a.rows, place(base + step));
}

template <typename T, int V, int E, int TPR>
__global__ void __launch_bounds__(kNormThreads<TPR>, TPR > 256 ? 2 : 4) gated_norm_fwd_kernel(const NormArgs a) {
    __shared__ float2 red[64];
    const Cols<V, E, TPR> cols{(int)threadIdx.x % TPR, a.D};
    RowSum<TPR> sum{red};
    float w[E];
    cols.param(w, a.w);
    Raw<T, V> nx[E / V], nz[E / V];
    auto fetch = [&](int64_t at) {
        cols.template fetch<T>(nx, a.x, at);
        cols.template fetch<T>(nz, a.z, at);
    };
    for_rows<TPR>(a, fetch, [] {}, [&](int64_t at, bool live, bool more, int64_t next) {
        float x[E], z[E];
        cols.template unpack<T>(x, nx);
        cols.template unpack<T>(z, nz);
        if (more) fetch(next);
        const float inv = rsqrtf(sum(dot(x, x)) / a.D + a.eps);
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = x[i] * inv * w[i] * act_value(z[i], a.silu);
        if (live) cols.template store<T>(a.y, at, x);
    });
}

// Column sums: in registers, or (16 elements per thread, where registers run out) in this
// thread's own words of shared memory.
template <int E, int TPR>
struct ColumnSums {
    static constexpr bool kShared = E > 8;
    float s[kShared ? 1 : E];
    float *mem;  // [E][kNormThreads<TPR>]
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < E; ++i) at(i) = 0.f;
    }
    __device__ __forceinline__ float &at(int i) {
        if constexpr (kShared)
            return mem[i * kNormThreads<TPR> + threadIdx.x];
        else
            return s[i];
    }
};
template <int E, int TPR>
constexpr int kSumWords = E > 8 ? E * kNormThreads<TPR> : 1;

// Adds the row groups' column sums in the order of the groups and writes them for this block.
template <int V, int E, int TPR>
__device__ __forceinline__ void store_column_sums(const Cols<V, E, TPR> &cols, ColumnSums<E, TPR> &s, float *out, float *buf) {
    if constexpr (kNormRows<TPR> == 1) {
#pragma unroll
        for (int k = 0; k < E / V; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (cols.in(k)) out[cols.col(k) + v] = s.at(k * V + v);
    } else {
        const int group = threadIdx.x / TPR;
        for (int g = 0; g < kNormRows<TPR>; ++g) {
            __syncthreads();
            if (g == group)
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    float *at = &buf[i * TPR + cols.lane];
                    *at = g == 0 ? s.at(i) : *at + s.at(i);
                }
        }
        __syncthreads();
        if (group == 0)
#pragma unroll
            for (int k = 0; k < E / V; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (cols.in(k)) out[cols.col(k) + v] = buf[(k * V + v) * TPR + cols.lane];
        __syncthreads();
    }
}
template <int E, int TPR>
constexpr int kGroupWords = kNormRows<TPR> > 1 ? E * TPR : 1;

template <typename T, int V, int E, int TPR>
__global__ void __launch_bounds__(kNormThreads<TPR>, TPR > 256 ? 1 : 3) gated_norm_bwd_kernel(const NormArgs a) {
    extern __shared__ float dyn[];
    __shared__ float2 red[64];
    __shared__ float buf[kGroupWords<E, TPR>];
    const Cols<V, E, TPR> cols{(int)threadIdx.x % TPR, a.D};
    RowSum<TPR> sum{red};
    ColumnSums<E, TPR> dw;
    dw.mem = dyn;
    dw.zero();
    float w[E];
    cols.param(w, a.w);
    Raw<T, V> nx[E / V], nz[E / V], ndy[E / V];
    auto fetch = [&](int64_t at) {
        cols.template fetch<T>(nx, a.x, at);
        cols.template fetch<T>(nz, a.z, at);
        cols.template fetch<T>(ndy, a.dy, at);
    };
    for_rows<TPR>(a, fetch, [] {}, [&](int64_t at, bool live, bool more, int64_t next) {
        float x[E], z[E], g[E], der[E];
        cols.template unpack<T>(x, nx);
        cols.template unpack<T>(z, nz);
        cols.template unpack<T>(g, ndy);
        if (more) fetch(next);
#pragma unroll
        for (int i = 0; i < E; ++i) {
            float val;
            act_both(z[i], a.silu, val, der[i]);
            der[i] *= g[i] * w[i];  // times n: the gradient of z
            z[i] = g[i] * val;      // times n: the gradient of the weight
            g[i] = z[i] * w[i];     // the gradient of n
        }
        const float2 t = sum(dot(x, x), dot(g, x));
        const float inv = rsqrtf(t.x / a.D + a.eps), m = inv * t.y / a.D;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float n = x[i] * inv;
            if (live) dw.at(i) = fmaf(z[i], n, dw.at(i));
            der[i] *= n;
            x[i] = inv * fmaf(-n, m, g[i]);
        }
        if (live) {
            cols.template store<T>(a.dz, at, der);
            cols.template store<T>(a.dx, at, x);
        }
    });
    store_column_sums(cols, dw, a.partial + (int64_t)blockIdx.x * a.D, buf);
}

// The block norm's parameters of a row group in shared memory: weight, and post_weight scale (what
// multiplies n act(z) in r'). Registers do not hold them beside a row, and from memory they would be
// fetched behind the next row's loads (216 against 180 us for the gradient of 8192 x 4096 when this was chosen).
template <int V, int E, int TPR>
struct BlockParams {
    float *w, *f;
    __device__ __forceinline__ BlockParams(const Cols<V, E, TPR> &cols, const NormArgs &a, float *mem) {
        w = mem;
        f = mem + E * TPR;
        if (threadIdx.x < TPR) {
            float t[E], u[E];
            cols.param(t, a.w);
            cols.keep(w, t);
            cols.param(t, a.pw);
            cols.param(u, a.scale);
#pragma unroll
            for (int i = 0; i < E; ++i) t[i] *= u[i];
            cols.keep(f, t);
        }
        __syncthreads();
    }
};

// R: the residual's type.
template <typename T, typename R, int V, int E, int TPR>
__global__ void __launch_bounds__(kNormThreads<TPR>, TPR > 256 ? 2 : 4) block_norm_fwd_kernel(const NormArgs a) {
    extern __shared__ __align__(16) float dyn[];
    __shared__ float2 red[64];
    const Cols<V, E, TPR> cols{(int)threadIdx.x % TPR, a.D};
    const BlockParams<V, E, TPR> par(cols, a, dyn);
    RowSum<TPR> sum{red};
    Raw<T, V> nx[E / V], nz[E / V];
    Raw<R, V> nr[E / V];
    auto fetch = [&](int64_t at) {
        cols.template fetch<T>(nx, a.x, at);
        cols.template fetch<R>(nr, a.res, at);
        if (a.z != nullptr) cols.template fetch<T>(nz, a.z, at);
    };
    for_rows<TPR>(a, fetch, [] {}, [&](int64_t at, bool live, bool more, int64_t next) {
        float x[E], r[E], t[E];
        cols.template unpack<T>(x, nx);
        cols.template unpack<R>(r, nr);
        if (a.z != nullptr) cols.template unpack<T>(t, nz);
        // r is written before the next row is read: the update in place stays within a row
        if (more) fetch(next);
        float inv = 1.f;
        if (a.pw != nullptr) inv = rsqrtf(sum(dot(x, x)) / a.D + a.eps);
        if (a.z != nullptr) {
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] *= act_value(t[i], a.silu);
        }
        cols.own(t, par.f);
#pragma unroll
        for (int i = 0; i < E; ++i) r[i] = fmaf(x[i], inv * t[i], r[i]);
        if (live) cols.template store<R>(a.nres, at, r);
        cols.own(t, par.w);
        const float rinv = rsqrtf(sum(dot(r, r)) / a.D + a.eps);
#pragma unroll
        for (int i = 0; i < E; ++i) r[i] *= rinv * t[i];
        if (live) cols.template store<T>(a.y, at, r);
    });
}

template <typename T, typename R, int V, int E, int TPR>
__global__ void __launch_bounds__(kNormThreads<TPR>, TPR > 256 ? 1 : 2) block_norm_bwd_kernel(const NormArgs a) {
    extern __shared__ __align__(16) float dyn[];
    __shared__ float2 red[64];
    __shared__ float buf[kGroupWords<E, TPR>];
    constexpr bool kAhead = E <= 8;  // the next row's loads ahead: registers allow it for 8 elements
    const Cols<V, E, TPR> cols{(int)threadIdx.x % TPR, a.D};
    RowSum<TPR> sum{red};
    const BlockParams<V, E, TPR> par(cols, a, dyn);
    // dw; and sum of dr' act(z) n, from which dscale = post_weight x it, dpost_weight = scale x it
    ColumnSums<E, TPR> dw, dan;
    dw.mem = dyn + 2 * E * TPR;
    dan.mem = dw.mem + kSumWords<E, TPR>;
    dw.zero();
    dan.zero();
    Raw<T, V> nx[E / V], nz[E / V], ndy[E / V];
    Raw<R, V> nr[E / V], ndr[E / V];
    auto fetch_now = [&](int64_t at) {
        cols.template fetch<T>(nx, a.x, at);
        cols.template fetch<R>(nr, a.res, at);
        if (a.z != nullptr) cols.template fetch<T>(nz, a.z, at);
        cols.template fetch<T>(ndy, a.dy, at);
        if (a.dres != nullptr) cols.template fetch<R>(ndr, a.dres, at);
    };
    auto fetch = [&](int64_t at) {
        if (kAhead) fetch_now(at);
    };
    float xx = 0.f;  // sum of x^2 over the row whose turn is next, from the turn before
    auto square = [&]() {
        float x[E];
        cols.template unpack<T>(x, nx);
        return dot(x, x);
    };
    auto before = [&]() {
        if (kAhead && a.pw != nullptr) xx = sum(square());
    };
    for_rows<TPR>(a, fetch, before, [&](int64_t at, bool live, bool more, int64_t next) {
        if (!kAhead) fetch_now(at);
        float n[E], r[E], z[E], g[E], t[E], dr[E];
        cols.template unpack<T>(n, nx);
        cols.template unpack<R>(r, nr);
        if (a.z != nullptr) cols.template unpack<T>(z, nz);
        cols.template unpack<T>(t, ndy);
        if (a.dres != nullptr) {
            cols.template unpack<R>(dr, ndr);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) dr[i] = 0.f;
        }
        if (more) fetch(next);
        // the forward pass again: n = x / rms (or x), r = r'; g = scale act(z) post_weight
        float inv = 1.f;
        if (a.pw != nullptr) {
            inv = rsqrtf((kAhead ? xx : sum(dot(n, n))) / a.D + a.eps);
#pragma unroll
            for (int i = 0; i < E; ++i) n[i] *= inv;
        }
        float p[E];
        cols.own(g, par.f);
        float sg[E];  // sigmoid(z)
        if (a.z != nullptr) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                sg[i] = sigmoid(z[i]);
                r[i] = fmaf(g[i] * (a.silu ? z[i] * sg[i] : sg[i]), n[i], r[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                sg[i] = 1.f;
                r[i] = fmaf(g[i], n[i], r[i]);
            }
        }
        cols.own(p, par.w);
#pragma unroll
        for (int i = 0; i < E; ++i) p[i] *= t[i];  // dy weight
        const float2 q = sum(dot(r, r), dot(p, r));
        const float rinv = rsqrtf(q.x / a.D + a.eps), m = rinv * rinv * q.y / a.D;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (live) dw.at(i) = fmaf(t[i], r[i] * rinv, dw.at(i));
            dr[i] = fmaf(rinv, fmaf(-r[i], m, p[i]), dr[i]);  // gradient of r'
        }
        if (live) cols.template store<R>(a.dr, at, dr);
#pragma unroll
        for (int i = 0; i < E; ++i) {
            float val = sg[i], der = sg[i] * (1.f - sg[i]);  // without z: 1 and 0
            if (a.silu && a.z != nullptr) {
                der = fmaf(z[i], der, sg[i]);
                val = z[i] * sg[i];
            }
            const float tn = dr[i] * n[i];
            z[i] = tn * g[i] * der;
            if (live) dan.at(i) = fmaf(tn, val, dan.at(i));
            g[i] *= dr[i] * val;  // gradient of n
        }
        if (live && a.dz != nullptr) cols.template store<T>(a.dz, at, z);
        if (a.pw != nullptr) {
            float mn = dot(g, n);
            if (kAhead && more) {
                const float2 both = sum(mn, square());
                mn = both.x / a.D;
                xx = both.y;
            } else {
                mn = sum(mn) / a.D;
            }
#pragma unroll
            for (int i = 0; i < E; ++i) g[i] = inv * fmaf(-n[i], mn, g[i]);
        }
        if (live) cols.template store<T>(a.dx, at, g);
    });
    float *part = a.partial + (int64_t)blockIdx.x * 3 * a.D;
    store_column_sums(cols, dw, part, buf);
    ColumnSums<E, TPR> &d2 = dw;  // free now
    float pw[E], sc[E];
    cols.param(pw, a.pw);
    cols.param(sc, a.scale);
#pragma unroll
    for (int i = 0; i < E; ++i) d2.at(i) = sc[i] * dan.at(i);
    store_column_sums(cols, d2, part + a.D, buf);
#pragma unroll
    for (int i = 0; i < E; ++i) d2.at(i) = pw[i] * dan.at(i);
    store_column_sums(cols, d2, part + 2 * (int64_t)a.D, buf);
}

// ---- host -----------------------------------------------------------------------------------
struct NormPlan {
    int V, E, tpr;
    int64_t blocks;
};

// Threads and elements per row: 8 elements per thread (16 above 4096 channels), so as many threads as the row
// needs. They lie in vectors where every row of every tensor starts on 16 bytes; single channels
// otherwise, in three sizes only. `wide`: vectors of 8 channels, else of 4. Eight suit bf16 (16
// bytes). With fp32 tensors four let neighbouring threads read neighbouring 16 bytes, which the block norm's
// gradient gains from (8192 x 4096, fp32 residual: 145 -> 140 us) and its forward pass, already at
// the memory's rate, does not (16384 x 4096: 161 us with four, 144 with eight).
NormPlan norm_plan(int64_t rows, int D, bool vec, bool block, bool wide, int per_sm) {
    NormPlan q{};
    q.V = !vec ? 1 : (wide ? 8 : 4);
    q.E = D <= (vec ? 4096 : 1024) ? 8 : 16;
    if (!vec) {
        q.tpr = D <= 256 ? 32 : (D <= 1024 ? 128 : 512);
    } else {
        q.tpr = block ? 32 : 8;
        while (q.tpr < 512 && q.tpr * 8 < D) q.tpr *= 2;
    }
    const int per_block = q.tpr > 256 ? 1 : 256 / q.tpr;
    const int64_t most = (int64_t)(q.tpr > 256 ? (per_sm + 1) / 2 : per_sm) * (sm_count() > 0 ? sm_count() : 1);
    q.blocks = ceil_div(rows, per_block);
    if (q.blocks > most) q.blocks = most;
    if (q.blocks < 1) q.blocks = 1;
    return q;
}

// Runs a kernel; `params`: rows of parameters, `sums`: column sums (16 elements per thread only) that it
// keeps in shared memory.
template <int E, int TPR, typename K>
cudaError_t norm_run(K kernel, const NormPlan &q, const NormArgs &a, int params, int sums, cudaStream_t stream) {
    const size_t smem = ((size_t)params * E * TPR + (E > 8 ? (size_t)sums * kSumWords<E, TPR> : 0)) * sizeof(float);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    kernel<<<(unsigned)q.blocks, kNormThreads<TPR>, smem, stream>>>(a);
    return cudaGetLastError();
}

#define KDA_NORM_LAUNCH(kernel, params, sums, V_, E_, TPR_, ...) \
    if (q.V == V_ && q.E == E_ && q.tpr == TPR_) return norm_run<E_, TPR_>(kernel<__VA_ARGS__, V_, E_, TPR_>, q, a, params, sums, stream);
#define KDA_NORM_BLOCK_SIZES(kernel, params, sums, V_, ...) \
    KDA_NORM_LAUNCH(kernel, params, sums, V_, 8, 32, __VA_ARGS__) \
    KDA_NORM_LAUNCH(kernel, params, sums, V_, 8, 64, __VA_ARGS__) \
    KDA_NORM_LAUNCH(kernel, params, sums, V_, 8, 128, __VA_ARGS__) \
    KDA_NORM_LAUNCH(kernel, params, sums, V_, 8, 256, __VA_ARGS__) \
    KDA_NORM_LAUNCH(kernel, params, sums, V_, 8, 512, __VA_ARGS__) \
    KDA_NORM_LAUNCH(kernel, params, sums, V_, 16, 512, __VA_ARGS__) \
    KDA_NORM_LAUNCH(kernel, params, sums, 1, 8, 32, __VA_ARGS__) \
    KDA_NORM_LAUNCH(kernel, params, sums, 1, 8, 128, __VA_ARGS__) \
    KDA_NORM_LAUNCH(kernel, params, sums, 1, 16, 512, __VA_ARGS__)
#define KDA_NORM_GATED_SIZES(kernel, params, sums, V_, ...) \
    KDA_NORM_LAUNCH(kernel, params, sums, V_, 8, 8, __VA_ARGS__) \
    KDA_NORM_LAUNCH(kernel, params, sums, V_, 8, 16, __VA_ARGS__) \
    KDA_NORM_BLOCK_SIZES(kernel, params, sums, V_, __VA_ARGS__)

template <typename T>
cudaError_t launch_gated(const NormPlan &q, const NormArgs &a, bool bwd, cudaStream_t stream) {
    constexpr int V = sizeof(T) == 2 ? 8 : 4;
    if (bwd) {
        KDA_NORM_GATED_SIZES(gated_norm_bwd_kernel, 0, 1, V, T)
    } else {
        KDA_NORM_GATED_SIZES(gated_norm_fwd_kernel, 0, 0, V, T)
    }
    return cudaErrorInvalidValue;
}
template <typename T, typename R>
cudaError_t launch_block(const NormPlan &q, const NormArgs &a, bool bwd, cudaStream_t stream) {
    if (bwd) {
        KDA_NORM_BLOCK_SIZES(block_norm_bwd_kernel, 2, 2, 4, T, R)
    } else {
        KDA_NORM_BLOCK_SIZES(block_norm_fwd_kernel, 2, 0, 8, T, R)
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
    const void *ptrs[] = {p.f.x, p.f.z, p.dy, p.dx, p.dz, p.f.weight};
    return norm_plan(p.f.rows, p.f.D, vec_ok(p.f.D, ptrs, 6), false, p.f.dtype == KDA_DTYPE_BF16, 3);
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
    const void *ptrs[] = {p.f.x, p.f.z, p.f.residual, p.dy, p.dres, p.dx, p.dresidual, p.dz, p.f.weight, p.f.post_weight, p.f.scale};
    return norm_plan(p.f.rows, p.f.D, vec_ok(p.f.D, ptrs, 11), true, false, 2);
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
    const void *ptrs[] = {p->x, p->z, p->y, p->weight};
    const NormPlan q = norm_plan(p->rows, p->D, vec_ok(p->D, ptrs, 4), false, p->dtype == KDA_DTYPE_BF16, 4);
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
    const void *ptrs[] = {p->x, p->z, p->residual, p->y, p->new_residual, p->weight, p->post_weight, p->scale};
    const NormPlan q = norm_plan(p->rows, p->D, vec_ok(p->D, ptrs, 8), true, true, 16);
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
