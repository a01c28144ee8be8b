// Short causal depthwise convolution and its gradient (kda_mixer.h: kda_conv_*).
//
//   y_t = act(b + sum_j w_j x_{t-W+1+j}),   W = 2..4 taps per channel,
//
// x before a sequence's first token being its initial state. One thread takes four neighbouring
// channels (one where rows are not aligned for that) through a tile of rows with the last W - 1 inputs in registers, so that each
// input is read once (plus W - 1 rows per tile) and every access is four contiguous elements.
// Tiles are cut over the rows of all sequences together: where a sequence ends inside
// a tile its window is refilled from the next one's initial state, so ragged packed batches need
// no table of tiles.
//
// Bound by memory: 2 bytes in and 2 out per bf16 element. 32761 packed rows of 8192 channels in bf16: 174 us,
// 6.2 TB/s. The gradient (16384 x 12288: 250 us, 4.8 TB/s) also issues 29 instructions per element.
#include "mixer_common.cuh"

namespace kda {
namespace {

using namespace mix;

constexpr int kConvThreads = 128;

struct ConvArgs {
    const void *x;
    const float *w, *bias;
    const void *s0;
    void *y, *st;
    const void *dy, *dst;
    void *dx, *ds0;
    float *partial;  // per tile: dweight [D][W], then dbias [D]
    int64_t xs;      // elements between rows of x
    int D, tile, silu;
    int wvec;        // weight on 16 bytes
    int64_t tiles;
    Seqs seqs;
    unsigned int *err;
};

// V channels as pairs (or a single one): one instruction does a multiply-add for two channels.
template <int V>
struct Lanes {
    using type = f2;
    static constexpr int K = V / 2;
};
template <>
struct Lanes<1> {
    using type = float;
    static constexpr int K = 1;
};
__device__ __forceinline__ float fma_(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ f2 fma_(f2 a, f2 b, f2 c) { return fma2(a, b, c); }
__device__ __forceinline__ float mul_(float a, float b) { return a * b; }
__device__ __forceinline__ f2 mul_(f2 a, f2 b) { return mul2(a, b); }
__device__ __forceinline__ float add_(float a, float b) { return a + b; }
__device__ __forceinline__ f2 add_(f2 a, f2 b) { return add2(a, b); }
__device__ __forceinline__ float silu_(float s) { return s * sigmoid(s); }
__device__ __forceinline__ f2 silu_(f2 s) {
    float a, b;
    upk(s, a, b);
    return pk(silu_(a), silu_(b));
}
// silu'(s) = p (1 + s (1 - p)), p = 1 / (1 + e^-s)
__device__ __forceinline__ float dsilu_(float s) {
    const float p = sigmoid(s);
    return fmaf(fmaf(-p, s, s), p, p);
}
__device__ __forceinline__ f2 dsilu_(f2 s) {
    float a, b;
    upk(s, a, b);
    return pk(dsilu_(a), dsilu_(b));
}

template <typename T, int V>
struct Row {
    using L = typename Lanes<V>::type;
    static constexpr int K = Lanes<V>::K;
    L v[K];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = 0;
    }
    __device__ __forceinline__ void from(const Raw<T, V> &r) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if constexpr (V > 1)
                v[k] = r.pair(k);
            else
                v[k] = r.get(k);
        }
    }
    __device__ __forceinline__ void floats(float (&f)[V]) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if constexpr (V > 1)
                upk(v[k], f[2 * k], f[2 * k + 1]);
            else
                f[k] = v[k];
        }
    }
    __device__ __forceinline__ void set(const float (&f)[V]) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if constexpr (V > 1)
                v[k] = pk(f[2 * k], f[2 * k + 1]);
            else
                v[k] = f[k];
        }
    }
    __device__ __forceinline__ void load(const T *p) {
        Raw<T, V> r;
        r.load(p);
        from(r);
    }
    __device__ __forceinline__ void store(T *p) const {
        float f[V];
        floats(f);
        store_vec<T, V>(p, f);
    }
};
// a += b c
template <typename T, int V>
__device__ __forceinline__ void mad(Row<T, V> &a, const Row<T, V> &b, const Row<T, V> &c) {
#pragma unroll
    for (int k = 0; k < Row<T, V>::K; ++k) a.v[k] = fma_(b.v[k], c.v[k], a.v[k]);
}

// The taps and the bias of V channels.
template <typename T, int V, int W>
__device__ __forceinline__ void load_weights(const ConvArgs &a, uint32_t c, Row<T, V> (&w)[W], Row<T, V> &b) {
    float f[V * W], fb[V];
    if (V > 1 && a.wvec) {
#pragma unroll
        for (int i = 0; i < V * W / 4; ++i) {
            const float4 q = reinterpret_cast<const float4 *>(a.w + (int64_t)c * W)[i];
            f[4 * i] = q.x;
            f[4 * i + 1] = q.y;
            f[4 * i + 2] = q.z;
            f[4 * i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V * W; ++i) f[i] = a.w[(int64_t)c * W + i];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) fb[v] = a.bias != nullptr ? a.bias[c + v] : 0.f;
    b.set(fb);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float t[V];
#pragma unroll
        for (int v = 0; v < V; ++v) t[v] = f[v * W + j];
        w[j].set(t);
    }
}

// The window before row r of a sequence: rows r - (W-1) .. r - 1, those before the sequence's
// start from its initial state.
template <typename T, int V, int W>
__device__ __forceinline__ void fill_window(const ConvArgs &a, const SeqAt &at, int64_t r, uint32_t c, Row<T, V> (&win)[W]) {
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        const int64_t pos = r - (W - 1) + i;
        const int64_t slot = W - 1 + pos - at.start;  // >= 0 since r >= start
        if (pos >= at.start)
            win[i].load(static_cast<const T *>(a.x) + pos * a.xs + c);
        else if (a.s0 != nullptr)
            win[i].load(static_cast<const T *>(a.s0) + ((int64_t)at.s * (W - 1) + slot) * a.D + c);
        else
            win[i].zero();
    }
}

template <typename T, int V>
__device__ __forceinline__ void copy_state(const void *from, void *to, int64_t at) {
    Raw<T, V> r;
    if (from != nullptr)
        r.load(static_cast<const T *>(from) + at);
    else
        r.zero();
    r.store(static_cast<T *>(to) + at);
}

// Rows that are loaded together, while the previous ones are worked on; inside a sequence and a tile they
// are also worked on together, without a check or a move per row. Blocks per SM (registers) go with
// that: what keeps the memory busy is rows in flight times blocks.
template <typename T>
constexpr int kFwdBatch = sizeof(T) == 2 ? 8 : 4;
constexpr int kBwdBatch = 4;
constexpr int kFwdPerSM = 5;  // 32761 x 8192 bf16: 174 us; six blocks 192, four rows and eight blocks 181
template <typename T>
constexpr int kBwdPerSM = sizeof(T) == 2 ? 4 : 3;  // 16384 x 12288 bf16: 250 us; five blocks spill (500), three with 8 rows 283

template <typename T, int V, int W, bool SILU>
__global__ void __launch_bounds__(kConvThreads, kFwdPerSM) conv_fwd_kernel(const ConvArgs a) {
    constexpr int kBatch = kFwdBatch<T>;
    using R = Row<T, V>;
    if (blockIdx.x == 0 && blockIdx.y == 0) seq_check(a.seqs, a.err, threadIdx.x, kConvThreads);
    // 32 bits without a sign: a row's place is the same for all threads, and the thread's own part of an
    // address then needs no 64-bit arithmetic
    const uint32_t c = (blockIdx.y * kConvThreads + threadIdx.x) * V;
    if (c >= (uint32_t)a.D) return;
    // empty sequences keep their state; the tiles share them out
    if (a.st != nullptr)
        for (int64_t s = blockIdx.x; s < a.seqs.N; s += gridDim.x)
            if (seq_empty(a.seqs, (int)s)) {
#pragma unroll
                for (int i = 0; i < W - 1; ++i) copy_state<T, V>(a.s0, a.st, (s * (W - 1) + i) * a.D + c);
            }
    const int64_t r0 = (int64_t)blockIdx.x * a.tile;
    const int64_t r1 = r0 + a.tile < a.seqs.rows ? r0 + a.tile : a.seqs.rows;
    if (r0 >= r1) return;

    R w[W], b, win[W];
    load_weights<T, V, W>(a, c, w, b);
    SeqAt at = seq_find(a.seqs, r0);
    fill_window<T, V, W>(a, at, r0, c, win);

    Raw<T, V> next[kBatch];
    auto fetch = [&](int64_t rb) {
        const T *x = static_cast<const T *>(a.x) + rb * a.xs;  // the same for all threads
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (rb + i < r1) next[i].load(x + i * a.xs + c);
    };
    auto put = [&](int64_t r, R s) {
        if (SILU)
#pragma unroll
            for (int k = 0; k < R::K; ++k) s.v[k] = silu_(s.v[k]);
        s.store(static_cast<T *>(a.y) + r * a.D + c);
    };
    auto keep_state = [&]() {
        T *st = static_cast<T *>(a.st) + (int64_t)at.s * (W - 1) * a.D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[j].store(st + (int64_t)j * a.D);
    };
    fetch(r0);
    for (int64_t rb = r0; rb < r1; rb += kBatch) {
        Raw<T, V> in[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) in[i] = next[i];
        if (rb + kBatch < r1) fetch(rb + kBatch);
        if (rb + kBatch <= r1 && rb + kBatch <= at.end) {
            R ext[W - 1 + kBatch];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) ext[j] = win[j];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                ext[W - 1 + i].from(in[i]);
                R s = b;
#pragma unroll
                for (int j = 0; j < W; ++j) mad(s, w[j], ext[i + j]);
                put(rb + i, s);
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j) win[j] = ext[kBatch + j];
            if (rb + kBatch == at.end && a.st != nullptr) keep_state();
        } else {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int64_t r = rb + i;
                if (r >= r1) break;
                if (r == at.end) {
                    seq_next(a.seqs, at);
                    fill_window<T, V, W>(a, at, r, c, win);
                }
                win[W - 1].from(in[i]);
                R s = b;
#pragma unroll
                for (int j = 0; j < W; ++j) mad(s, w[j], win[j]);
                put(r, s);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) win[j] = win[j + 1];
                if (r + 1 == at.end && a.st != nullptr) keep_state();
            }
        }
    }
}

// Gradient. With p_t the sum before the activation and g_t = dy_t act'(p_t),
//   dx_p = sum_k g_{p+k} w_{W-1-k}   over the tokens p + k of the same sequence,
//   dw_j = sum_t g_t x_{t-W+1+j},  db = sum_t g_t,
// and the same sum gives ds0 at the W - 1 positions before the sequence; dst is added at
// the positions that the final state holds. The thread walks its tile and W - 1 rows more with
// the windows of x and g in registers and finishes position q - (W-1) at row q; where
// a sequence ends, the open positions are finished with zeros.
template <typename T, int V, int W>
struct ConvBack {
    using R = Row<T, V>;
    const ConvArgs &a;
    uint32_t c;
    int64_t r0, r1;
    R w[W], g[W];

    __device__ __forceinline__ ConvBack(const ConvArgs &args) : a(args) {}
    __device__ __forceinline__ void shift() {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) g[j] = g[j + 1];
    }
    // finish position p; `slot` of the final state holds it when slot >= 0
    __device__ __forceinline__ void finish(const SeqAt &at, int64_t p, int slot) const {
        const bool token = p >= at.start;
        if (token ? (p < r0 || p >= r1) : (at.start < r0 || a.ds0 == nullptr)) return;
        R s;
        s.zero();
        if (slot >= 0 && a.dst != nullptr)
            s.load(static_cast<const T *>(a.dst) + ((int64_t)at.s * (W - 1) + slot) * a.D + c);
#pragma unroll
        for (int k = 0; k < W; ++k) mad(s, g[k], w[W - 1 - k]);
        s.store(token ? static_cast<T *>(a.dx) + p * a.D + c
                      : static_cast<T *>(a.ds0) + ((int64_t)at.s * (W - 1) + (W - 1 + p - at.start)) * a.D + c);
    }
    // the sequence has ended: its last W - 1 positions
    __device__ __forceinline__ void flush(const SeqAt &at) {
#pragma unroll
        for (int k = 1; k < W; ++k) {
            shift();
            g[W - 1].zero();
            finish(at, at.end - W + k, k - 1);
        }
#pragma unroll
        for (int j = 0; j < W; ++j) g[j].zero();
    }
};

template <typename T, int V, int W, bool SILU>
__global__ void __launch_bounds__(kConvThreads, kBwdPerSM<T>) conv_bwd_kernel(const ConvArgs a) {
    constexpr int kBatch = kBwdBatch;
    using R = Row<T, V>;
    if (blockIdx.x == 0 && blockIdx.y == 0) seq_check(a.seqs, a.err, threadIdx.x, kConvThreads);
    // 32 bits without a sign: a row's place is the same for all threads, and the thread's own part of an
    // address then needs no 64-bit arithmetic
    const uint32_t c = (blockIdx.y * kConvThreads + threadIdx.x) * V;
    if (c >= (uint32_t)a.D) return;
    if (a.ds0 != nullptr)
        for (int64_t s = blockIdx.x; s < a.seqs.N; s += gridDim.x)
            if (seq_empty(a.seqs, (int)s)) {
#pragma unroll
                for (int i = 0; i < W - 1; ++i) copy_state<T, V>(a.dst, a.ds0, (s * (W - 1) + i) * a.D + c);
            }
    ConvBack<T, V, W> k(a);
    k.c = c;
    k.r0 = (int64_t)blockIdx.x * a.tile;
    k.r1 = k.r0 + a.tile < a.seqs.rows ? k.r0 + a.tile : a.seqs.rows;
    R b, dw[W], db, win[W];
    load_weights<T, V, W>(a, c, k.w, b);
    db.zero();
#pragma unroll
    for (int j = 0; j < W; ++j) {
        dw[j].zero();
        k.g[j].zero();
    }
    if (k.r0 < k.r1) {
        const int64_t qend = k.r1 + W - 1 < a.seqs.rows ? k.r1 + W - 1 : a.seqs.rows;
        SeqAt at = seq_find(a.seqs, k.r0);
        fill_window<T, V, W>(a, at, k.r0, c, win);
        Raw<T, V> nx[kBatch], ng[kBatch];
        auto fetch = [&](int64_t qb) {
            const T *x = static_cast<const T *>(a.x) + qb * a.xs, *dy = static_cast<const T *>(a.dy) + qb * a.D;
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (qb + i < qend) {
                    nx[i].load(x + i * a.xs + c);
                    ng[i].load(dy + (int64_t)i * a.D + c);
                }
        };
        // g times the activation's derivative at the sum over the window `ext`
        auto before_act = [&](R &g, const R *ext) {
            if (!SILU) return;
            R s = b;
#pragma unroll
            for (int j = 0; j < W; ++j) mad(s, k.w[j], ext[j]);
#pragma unroll
            for (int i = 0; i < R::K; ++i) g.v[i] = mul_(g.v[i], dsilu_(s.v[i]));
        };
        auto add_weights = [&](const R &g, const R *ext) {
#pragma unroll
            for (int i = 0; i < R::K; ++i) db.v[i] = add_(db.v[i], g.v[i]);
#pragma unroll
            for (int j = 0; j < W; ++j) mad(dw[j], g, ext[j]);
        };
        bool open = true;  // false once the last sequence with rows in the tile has been finished
        fetch(k.r0);
        for (int64_t qb = k.r0; qb < qend && open; qb += kBatch) {
            Raw<T, V> in[kBatch], gr[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                in[i] = nx[i];
                gr[i] = ng[i];
            }
            if (qb + kBatch < qend) fetch(qb + kBatch);
            const int64_t p0 = qb - (W - 1);
            if (qb + kBatch <= k.r1 && qb + kBatch <= at.end && p0 >= at.start && p0 >= k.r0) {
                R ext[W - 1 + kBatch], gx[W - 1 + kBatch];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                    ext[j] = win[j];
                    gx[j] = k.g[j + 1];
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    ext[W - 1 + i].from(in[i]);
                    gx[W - 1 + i].from(gr[i]);
                    before_act(gx[W - 1 + i], ext + i);
                    add_weights(gx[W - 1 + i], ext + i);
                    R out;
                    out.zero();
#pragma unroll
                    for (int j = 0; j < W; ++j) mad(out, gx[i + j], k.w[W - 1 - j]);
                    out.store(static_cast<T *>(a.dx) + (p0 + i) * a.D + c);
                }
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                    win[j] = ext[kBatch + j];
                    k.g[j + 1] = gx[kBatch + j];
                }
                continue;
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int64_t q = qb + i;
                if (q >= qend || !open) break;
                if (q == at.end) {
                    k.flush(at);
                    if (q >= k.r1) {
                        open = false;
                        break;
                    }
                    seq_next(a.seqs, at);
                    fill_window<T, V, W>(a, at, q, c, win);
                }
                win[W - 1].from(in[i]);
                k.shift();
                k.g[W - 1].from(gr[i]);
                before_act(k.g[W - 1], win);
                if (q < k.r1) add_weights(k.g[W - 1], win);
                k.finish(at, q - (W - 1), -1);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) win[j] = win[j + 1];
            }
        }
        if (open && qend == at.end) k.flush(at);
    }
    float *part = a.partial + (int64_t)blockIdx.x * ((int64_t)a.D * (W + 1));
    float f[W][V], fb[V];
    db.floats(fb);
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j].floats(f[j]);
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) part[(int64_t)(c + v) * W + j] = f[j][v];
        part[(int64_t)a.D * W + c + v] = fb[v];
    }
}

template <typename T, int V, int W>
cudaError_t conv_launch(const ConvArgs &a, bool bwd, cudaStream_t stream) {
    const dim3 grid((unsigned)a.tiles, (unsigned)ceil_div(ceil_div(a.D, V), kConvThreads));
    if (bwd) {
        if (a.silu)
            conv_bwd_kernel<T, V, W, true><<<grid, kConvThreads, 0, stream>>>(a);
        else
            conv_bwd_kernel<T, V, W, false><<<grid, kConvThreads, 0, stream>>>(a);
    } else if (a.silu) {
        conv_fwd_kernel<T, V, W, true><<<grid, kConvThreads, 0, stream>>>(a);
    } else {
        conv_fwd_kernel<T, V, W, false><<<grid, kConvThreads, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t conv_width(const ConvArgs &a, int W, bool bwd, cudaStream_t stream) {
    if (W == 4) return conv_launch<T, V, 4>(a, bwd, stream);
    if (W == 3) return conv_launch<T, V, 3>(a, bwd, stream);
    return conv_launch<T, V, 2>(a, bwd, stream);
}

cudaError_t conv_dispatch(const ConvArgs &a, int dtype, int W, bool bwd, int V, cudaStream_t stream) {
    if (dtype == KDA_DTYPE_BF16) return V == 4 ? conv_width<bf16, 4>(a, W, bwd, stream) : conv_width<bf16, 1>(a, W, bwd, stream);
    return V == 4 ? conv_width<float, 4>(a, W, bwd, stream) : conv_width<float, 1>(a, W, bwd, stream);
}

int elem_size(int dtype) { return dtype == KDA_DTYPE_BF16 ? 2 : 4; }

// Checks shared by the three entry points.
int conv_check(const void *x, const float *weight, const float *bias, const void *s0, int64_t stride, int B, int T, int D, int W,
               const int32_t *cu, int dtype, int activation) {
    if (B < 1 || T < 0 || D < 1 || stride < 0 || (stride != 0 && stride < D)) return KDA_ERR_INVALID_ARG;
    if (weight == nullptr || (T != 0 && x == nullptr)) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_F32) return KDA_ERR_UNSUPPORTED;
    if (W < 2 || W > 4 || (activation != KDA_ACT_NONE && activation != KDA_ACT_SILU)) return KDA_ERR_UNSUPPORTED;
    const int e = elem_size(dtype);
    if (!aligned(x, e) || !aligned(s0, e) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(cu, 4)) return KDA_ERR_ALIGNMENT;
    const int64_t rows = cu != nullptr ? (int64_t)T : (int64_t)B * T;
    if (rows > INT32_MAX || ceil_div(D, kConvThreads) > 65535) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// Four channels per thread where every row of every tensor lets them be read at once, else one. (Eight
// channels take so many registers that they spill at five blocks per SM: 300 us for 32761 x 8192
// where four take 174.)
int conv_vec(int dtype, int D, int64_t xs, const void *const *ptrs, int n) {
    bool ok = D % 4 == 0 && xs % 4 == 0;
    for (int i = 0; i < n; ++i) ok = ok && aligned(ptrs[i], (size_t)4 * elem_size(dtype));
    return ok ? 4 : 1;
}

// Rows per tile: the tiles fill the GPU's slots (per_sm blocks per SM) `turns` times, or fewer
// times where tiles would get shorter than 32 rows (the W - 1 rows that two tiles both read, and a tile's
// first loads, then weigh more); where even one turn is not filled, tiles of at least 8 rows.
int conv_tile(int64_t rows, int64_t chan_blocks, int per_sm, int turns, int batch) {
    const int64_t slots = (int64_t)per_sm * (sm_count() > 0 ? sm_count() : 1);
    int64_t tile = 0;
    for (int t = turns; t >= 1 && tile < 32; --t) {
        const int64_t n = t * slots / chan_blocks;
        tile = ceil_div(ceil_div(rows, n < 1 ? 1 : n), batch) * batch;
    }
    return (int)(tile < 8 ? 8 : tile);
}

int conv_run(const kda_conv_params &p, bool step, cudaStream_t stream) {
    int st = conv_check(p.x, p.weight, p.bias, p.s0, p.x_stride, p.B, p.T, p.D, p.W, p.cu_seqlens, p.dtype, p.activation);
    if (st != KDA_OK) return st;
    if (p.T != 0 && p.y == nullptr) return KDA_ERR_INVALID_ARG;
    if (step && (p.cu_seqlens != nullptr || p.s0 == nullptr || p.st == nullptr)) return KDA_ERR_INVALID_ARG;
    // a sequence's tiles read s0 and write st independently of each other
    if (!step && p.st != nullptr && p.st == p.s0) return KDA_ERR_INVALID_ARG;
    const int e = elem_size(p.dtype);
    if (!aligned(p.y, e) || !aligned(p.st, e)) return KDA_ERR_ALIGNMENT;
    ConvArgs a{};
    a.x = p.x;
    a.w = p.weight;
    a.bias = p.bias;
    a.s0 = p.s0;
    a.y = p.y;
    a.st = p.st;
    a.xs = p.x_stride != 0 ? p.x_stride : p.D;
    a.D = p.D;
    a.silu = p.activation == KDA_ACT_SILU;
    a.wvec = aligned(p.weight, 16);
    a.seqs = Seqs{p.cu_seqlens, p.B, p.T, p.cu_seqlens != nullptr ? (int64_t)p.T : (int64_t)p.B * p.T};
    const cudaError_t e1 = device_error_word(&a.err);
    if (e1 != cudaSuccess) return status_of_cuda(e1);
    const void *ptrs[] = {p.x, p.s0, p.y, p.st};
    const int V = conv_vec(p.dtype, p.D, a.xs, ptrs, 4);
    if (step) {
        a.tile = p.T > 0 ? p.T : 1;  // one sequence per tile: its state is read and written by the same threads
        a.tiles = p.B;
    } else {
        a.tile = conv_tile(a.seqs.rows, ceil_div(ceil_div(p.D, V), kConvThreads), kFwdPerSM, 3,
                           p.dtype == KDA_DTYPE_BF16 ? kFwdBatch<bf16> : kFwdBatch<float>);
        a.tiles = ceil_div(a.seqs.rows, a.tile);
        if (a.tiles < 1) a.tiles = 1;
    }
    return status_of_cuda(conv_dispatch(a, p.dtype, p.W, false, V, stream));
}

struct ConvBwdPlan {
    int V, tile;
    int64_t tiles;
    size_t bytes;
};
ConvBwdPlan conv_bwd_plan(const kda_conv_bwd_params &p) {
    ConvBwdPlan q;
    const void *ptrs[] = {p.x, p.s0, p.dy, p.dst, p.dx, p.ds0};
    const int64_t rows = p.cu_seqlens != nullptr ? (int64_t)p.T : (int64_t)p.B * p.T;
    q.V = conv_vec(p.dtype, p.D, p.x_stride != 0 ? p.x_stride : p.D, ptrs, 6);
    q.tile = conv_tile(rows, ceil_div(ceil_div(p.D, q.V), kConvThreads), 
                       p.dtype == KDA_DTYPE_BF16 ? kBwdPerSM<bf16> : kBwdPerSM<float>, 2, kBwdBatch);
    q.tiles = ceil_div(rows, q.tile);
    if (q.tiles < 1) q.tiles = 1;
    q.bytes = (size_t)q.tiles * p.D * (p.W + 1) * sizeof(float);
    return q;
}

int conv_bwd_check(const kda_conv_bwd_params &p) {
    int st = conv_check(p.x, p.weight, p.bias, p.s0, p.x_stride, p.B, p.T, p.D, p.W, p.cu_seqlens, p.dtype, p.activation);
    if (st != KDA_OK) return st;
    if (p.dweight == nullptr || (p.T != 0 && (p.dy == nullptr || p.dx == nullptr))) return KDA_ERR_INVALID_ARG;
    const int e = elem_size(p.dtype);
    if (!aligned(p.dy, e) || !aligned(p.dst, e) || !aligned(p.dx, e) || !aligned(p.ds0, e) || !aligned(p.dweight, 4) ||
        !aligned(p.dbias, 4))
        return KDA_ERR_ALIGNMENT;
    return KDA_OK;
}

}  // namespace
}  // namespace kda

extern "C" {

int kda_conv_fwd(const kda_conv_params *p, cudaStream_t stream) {
    return p == nullptr ? KDA_ERR_INVALID_ARG : kda::conv_run(*p, false, stream);
}

int kda_conv_step(const kda_conv_params *p, cudaStream_t stream) {
    return p == nullptr ? KDA_ERR_INVALID_ARG : kda::conv_run(*p, true, stream);
}

size_t kda_conv_bwd_workspace(const kda_conv_bwd_params *p) {
    return p == nullptr || kda::conv_bwd_check(*p) != KDA_OK ? 0 : kda::conv_bwd_plan(*p).bytes;
}

int kda_conv_bwd(const kda_conv_bwd_params *p, cudaStream_t stream) {
    using namespace kda;
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    const int st = conv_bwd_check(*p);
    if (st != KDA_OK) return st;
    const ConvBwdPlan q = conv_bwd_plan(*p);
    if (p->workspace != nullptr && p->workspace_bytes < q.bytes) return KDA_ERR_INVALID_ARG;
    if (!aligned(p->workspace, 16)) return KDA_ERR_ALIGNMENT;
    ConvArgs a{};
    a.x = p->x;
    a.w = p->weight;
    a.bias = p->bias;
    a.s0 = p->s0;
    a.dy = p->dy;
    a.dst = p->dst;
    a.dx = p->dx;
    a.ds0 = p->ds0;
    a.xs = p->x_stride != 0 ? p->x_stride : p->D;
    a.D = p->D;
    a.silu = p->activation == KDA_ACT_SILU;
    a.wvec = aligned(p->weight, 16);
    a.tile = q.tile;
    a.tiles = q.tiles;
    a.seqs = Seqs{p->cu_seqlens, p->B, p->T, p->cu_seqlens != nullptr ? (int64_t)p->T : (int64_t)p->B * p->T};
    cudaError_t e = device_error_word(&a.err);
    if (e != cudaSuccess) return status_of_cuda(e);
    Scratch ws;
    e = ws.get(p->workspace, q.bytes, stream);
    if (e != cudaSuccess) return status_of_cuda(e);
    a.partial = static_cast<float *>(ws.ptr);
    e = conv_dispatch(a, p->dtype, p->W, true, q.V, stream);
    if (e == cudaSuccess) {
        const SumOuts outs{{p->dweight, p->dbias, nullptr, nullptr}, {(int64_t)p->D * p->W, p->D, 0, 0}};
        e = launch_sum_partials(a.partial, q.tiles, (int64_t)p->D * (p->W + 1), outs, stream);
    }
    return status_of_cuda(ws.release(e));
}

}  // extern "C"
