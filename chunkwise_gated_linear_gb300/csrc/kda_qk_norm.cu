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

// ---- rows of whole vectors -------------------------------------------------------------------
// LPR lanes share a row, 16 channels each as two chunks of 8; a warp holds 32 / LPR rows (heads of one token) at a time
// and U such groups, of queries, keys or values alone, for one token after another: what belongs to the
// channels (weights, frequencies) is loaded once, the angles once per token, and each group's rows of the
// next token are on their way as soon as the current ones are unpacked.
constexpr int kVecWarps = 8;

struct Share {
    int part;   // 0 queries, 1 keys, 2 values
    int head0;  // first head
};
// The slices of heads of a token, `each` heads apiece: of queries, then keys, then values.
__host__ __device__ __forceinline__ int slices_of(int heads, int each) { return (heads + each - 1) / each; }
__device__ __forceinline__ Share share_of(const HeadArgs &a, int slice, int each) {
    const int nq = slices_of(a.Hq, each), nk = slices_of(a.Hk, each);
    if (slice < nq) return Share{0, slice * each};
    slice -= nq;
    if (slice < nk) return Share{1, slice * each};
    return Share{2, (slice - nk) * each};
}

// The lane's place in a row.
struct LaneAt {
    int o0, o1;      // first channels of its two chunks
    bool in, turns;  // within the row; its channels are turned (pair e: freq[8 j + e])
};
template <int LPR>
__device__ __forceinline__ LaneAt lane_at(const HeadArgs &a, int part, int j) {
    LaneAt l;
    l.in = 16 * j < a.D;
    l.turns = part < 2 && 16 * j < a.R;
    l.o0 = 16 * j;
    l.o1 = 16 * j + 8;
    if (l.turns && !a.pairs) {  // channels i and i + R / 2
        l.o0 = 8 * j;
        l.o1 = a.R / 2 + 8 * j;
    }
    return l;
}

template <typename T>
struct Two {
    Raw<T, 8> a, b;
    __device__ __forceinline__ void load(const void *base, int64_t at, const LaneAt &l, bool ok) {
        if (ok) {
            a.load(static_cast<const T *>(base) + at + l.o0);
            b.load(static_cast<const T *>(base) + at + l.o1);
        } else {
            a.zero();
            b.zero();
        }
    }
    __device__ __forceinline__ void unpack(float (&f)[16]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[i] = a.get(i);
            f[8 + i] = b.get(i);
        }
    }
    static __device__ __forceinline__ void store(void *base, int64_t at, const LaneAt &l, const float (&f)[16]) {
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = f[i];
        store_vec<T, 8>(static_cast<T *>(base) + at + l.o0, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = f[8 + i];
        store_vec<T, 8>(static_cast<T *>(base) + at + l.o1, t);
    }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The lane's 8 pairs by their angles; `sign` -1: back.
__device__ __forceinline__ void turn_pairs(float (&f)[16], const float (&c)[8], const float (&s)[8], bool pairs, float sign) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float sn = s[e] * sign;
        if (pairs) {
            const float x = f[2 * e], y = f[2 * e + 1];
            f[2 * e] = x * c[e] - y * sn;
            f[2 * e + 1] = y * c[e] + x * sn;
        } else {
            const float x = f[e], y = f[8 + e];
            f[e] = x * c[e] - y * sn;
            f[8 + e] = y * c[e] + x * sn;
        }
    }
}

// A token's sequence as a warp goes from one token to a later one.
struct TokenAt {
    SeqAt at{0, 0, 0};
    int len = 0;  // in the cache
    __device__ __forceinline__ RowAt row(const HeadArgs &a, int64_t row, bool places) {
        if (row >= at.end) {
            at = seq_find(a.seqs, row);
            if (a.cached) len = cache_len(a.cache, at.s);
        }
        RowAt r;
        r.page = -1;
        r.slot = 0;
        r.pos = (int)(row - at.start);
        if (a.cached) {
            r.pos += len - (int)(at.end - at.start);
            if (places && r.pos >= 0) r.page = cache_page(a.cache, at.s, r.pos, r.slot);
        }
        if (a.pos != nullptr) r.pos = a.pos[row];
        return r;
    }
};

template <int LPR>
__device__ __forceinline__ void vec_put_e4m3(const Cache &c, bool value, const float (&f)[16], const LaneAt &l, bool ok, int page, int head, int slot,
                                             int j) {
    float top = 0.f;
    bool inf = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        top = fmaxf(top, finite_abs(f[i]));
        inf |= fabsf(f[i]) == INFINITY;
    }
    if (inf) top = INFINITY;
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = row_exponent(top);  // 120 for an infinity
    const float unit = pow2(-e);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = e4m3_pair(f[4 * i] * unit, f[4 * i + 1] * unit) | e4m3_pair(f[4 * i + 2] * unit, f[4 * i + 3] * unit) << 16;
    if (!ok || page < 0) return;
    const int64_t row = cache_row(c, page, head, slot);
    uint8_t *to = static_cast<uint8_t *>(value ? c.v : c.k) + row * c.D;
    *reinterpret_cast<uint2 *>(to + l.o0) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2 *>(to + l.o1) = make_uint2(w[2], w[3]);
    if (j == 0) (value ? c.vs : c.ks)[cache_scale(c, page, head, slot)] = (uint8_t)(e + 127);
}

template <typename T, int LPR, int U>
__global__ void __launch_bounds__(32 * kVecWarps, 2) vec_rows_kernel(const __grid_constant__ HeadArgs a, int slices, int tokens) {
    constexpr int kAtOnce = 32 / LPR;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / LPR, j = lane % LPR;
    if (blockIdx.x == 0) seq_check(a.seqs, a.err, threadIdx.x, 32 * kVecWarps);
    const Share sh = share_of(a, blockIdx.x % slices, U * kAtOnce);
    const LaneAt l = lane_at<LPR>(a, sh.part, j);
    const int64_t first = (int64_t)(blockIdx.x / slices) * tokens + warp;
    int64_t stop = (int64_t)(blockIdx.x / slices + 1) * tokens;
    if (stop > a.seqs.rows) stop = a.seqs.rows;
    if (first >= stop) return;
    const bool isq = sh.part == 0, isv = sh.part == 2;
    const int heads = isq ? a.Hq : isv ? a.Hv : a.Hk;
    const void *in = isq ? a.q : isv ? a.v : a.k;
    void *out = isq ? a.q_out : isv ? nullptr : a.k_out;
    const int64_t stride = isq ? a.q_stride : isv ? a.v_stride : a.k_stride;
    const float *w = isq ? a.qw : isv ? nullptr : a.kw;
    Two<T> raw[U];
    auto ok = [&](int u) { return l.in && sh.head0 + u * kAtOnce + sub < heads; };
    const int64_t lane_in = (int64_t)(sh.head0 + sub) * a.D;
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u].load(in, first * stride + lane_in + u * kAtOnce * a.D, l, ok(u));
    float wt[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) wt[i] = 1.f;
    if (w != nullptr && l.in) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // parameters may be aligned to 4 bytes alone
            wt[i] = w[l.o0 + i];
            wt[8 + i] = w[l.o1 + i];
        }
    }
    int64_t freq[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) freq[e] = l.turns ? a.freq[8 * j + e] : 0;
    TokenAt at;
    const float inv_d = 1.f / (float)a.D;
#pragma unroll 1
    for (int64_t row = first; row < stop; row += kVecWarps) {
        RowAt r{0, -1, 0};
        if (a.R > 0 || a.cached) r = at.row(a, row, !isq);
        float c[8], s[8];
        if (l.turns) {
#pragma unroll
            for (int e = 0; e < 8; ++e) turn(freq[e], r.pos, c[e], s[e]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int head = sh.head0 + u * kAtOnce + sub;
            float f[16];
            raw[u].unpack(f);
            if (row + kVecWarps < stop) raw[u].load(in, (row + kVecWarps) * stride + lane_in + u * kAtOnce * a.D, l, ok(u));
            if (w != nullptr) {
                float q = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) q = fmaf(f[i], f[i], q);
                const float inv = rsqrtf(row_sum<LPR>(q) * inv_d + a.eps);
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] *= inv * wt[i];
            }
            if (l.turns) turn_pairs(f, c, s, a.pairs, 1.f);
            if (out != nullptr && ok(u)) Two<T>::store(out, (row * heads + head) * a.D, l, f);
            if (a.cached && !isq) {
                if (a.cache.ks != nullptr)
                    vec_put_e4m3<LPR>(a.cache, isv, f, l, ok(u), r.page, head, r.slot, j);
                else if (ok(u) && r.page >= 0)
                    Two<T>::store(isv ? a.cache.v : a.cache.k, cache_row(a.cache, r.page, head, r.slot) * a.D, l, f);
            }
        }
    }
}

template <typename T, int LPR, int U>
__global__ void __launch_bounds__(32 * kVecWarps, 2) vec_rows_bwd_kernel(const __grid_constant__ HeadArgs a, int slices, int tokens) {
    constexpr int kAtOnce = 32 / LPR;
    __shared__ float red[kVecWarps][kMaxD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / LPR, j = lane % LPR;
    if (blockIdx.x == 0) seq_check(a.seqs, a.err, threadIdx.x, 32 * kVecWarps);
    const Share sh = share_of(a, blockIdx.x % slices, U * kAtOnce);
    const LaneAt l = lane_at<LPR>(a, sh.part, j);
    const int64_t first = (int64_t)(blockIdx.x / slices) * tokens + warp;
    int64_t stop = (int64_t)(blockIdx.x / slices + 1) * tokens;
    if (stop > a.seqs.rows) stop = a.seqs.rows;
    const bool isq = sh.part == 0;
    const int heads = isq ? a.Hq : a.Hk;
    const void *in = isq ? a.q : a.k, *dout = isq ? a.dq_out : a.dk_out;
    void *out = isq ? a.q_out : a.k_out;
    const int64_t stride = isq ? a.q_stride : a.k_stride;
    const float *w = isq ? a.qw : a.kw;
    Two<T> raw[U], raw_g[U];
    auto ok = [&](int u) { return l.in && sh.head0 + u * kAtOnce + sub < heads; };
    auto fetch = [&](int u, int64_t row) {
        const int head = sh.head0 + u * kAtOnce + sub;
        raw_g[u].load(dout, (row * heads + head) * a.D, l, ok(u));
        if (w != nullptr) raw[u].load(in, row * stride + (int64_t)head * a.D, l, ok(u));
    };
    if (first < stop) {
#pragma unroll
        for (int u = 0; u < U; ++u) fetch(u, first);
    }
    float wt[16], sum[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        wt[i] = w != nullptr && l.in ? w[(i < 8 ? l.o0 : l.o1 - 8) + i] : 0.f;
        sum[i] = 0.f;
    }
    int64_t freq[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) freq[e] = l.turns ? a.freq[8 * j + e] : 0;
    TokenAt at;
    const float inv_d = 1.f / (float)a.D;
#pragma unroll 1
    for (int64_t row = first; row < stop; row += kVecWarps) {
        int pos = 0;
        if (a.R > 0) pos = at.row(a, row, false).pos;
        float c[8], s[8];
        if (l.turns) {
#pragma unroll
            for (int e = 0; e < 8; ++e) turn(freq[e], pos, c[e], s[e]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float g[16], x[16];
            raw_g[u].unpack(g);
            if (w != nullptr) raw[u].unpack(x);
            if (row + kVecWarps < stop) fetch(u, row + kVecWarps);
            if (l.turns) turn_pairs(g, c, s, a.pairs, -1.f);
            if (w != nullptr) {
                float q = 0.f, m = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    q = fmaf(x[i], x[i], q);
                    m = fmaf(g[i] * x[i], wt[i], m);
                }
                q = row_sum<LPR>(q);
                m = row_sum<LPR>(m);
                const float inv = rsqrtf(q * inv_d + a.eps);
                m *= inv_d * inv * inv;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    sum[i] = fmaf(g[i] * x[i], inv, sum[i]);
                    g[i] = inv * (g[i] * wt[i] - x[i] * m);
                }
            }
            if (ok(u)) Two<T>::store(out, (row * heads + sh.head0 + u * kAtOnce + sub) * a.D, l, g);
        }
    }
    if (a.partial == nullptr) return;
    // the weight's gradient of this block: over the rows of a warp, then its warps in order; zeros for the other weight
#pragma unroll
    for (int i = 0; i < 16; ++i) {
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
        if (sub == 0 && l.in) red[warp][(i < 8 ? l.o0 : l.o1 - 8) + i] = sum[i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.D; i += 32 * kVecWarps) {
        float t = 0.f;
        if ((i < a.D) == isq) {
#pragma unroll
            for (int v = 0; v < kVecWarps; ++v) t += red[v][i < a.D ? i : i - a.D];
        }
        a.partial[(int64_t)blockIdx.x * 2 * a.D + i] = t;
    }
}

// Rows of the cache into contiguous ones: a lane has 16 channels of a row.
template <typename T, int LPR, int U>
__global__ void __launch_bounds__(32 * kVecWarps) vec_read_kernel(const __grid_constant__ HeadArgs a, int slices, int tokens) {
    constexpr int kAtOnce = 32 / LPR;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / LPR, j = lane % LPR;
    const Cache &c = a.cache;
    if (blockIdx.x == 0) seq_check(a.seqs, a.err, threadIdx.x, 32 * kVecWarps);
    const int half = slices / 2, slice = blockIdx.x % slices;
    const bool isv = slice >= half;
    const int head0 = (isv ? slice - half : slice) * U * kAtOnce;
    const int64_t first = (int64_t)(blockIdx.x / slices) * tokens + warp;
    int64_t stop = (int64_t)(blockIdx.x / slices + 1) * tokens;
    if (stop > a.seqs.rows) stop = a.seqs.rows;
    const LaneAt l{16 * j, 16 * j + 8, 16 * j < c.D, false};
    void *out = isv ? a.q_out : a.k_out;
    const void *base = isv ? c.v : c.k;
    TokenAt at;
#pragma unroll 1
    for (int64_t row = first; row < stop; row += kVecWarps) {
        const RowAt r = at.row(a, row, true);
        uint4 q[U];
        uint32_t e[U];
        Two<T> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int head = head0 + u * kAtOnce + sub;
            const bool ok = l.in && head < a.Hk && r.page >= 0;
            const int64_t from = ok ? cache_row(c, r.page, head, r.slot) : 0;
            if (c.ks != nullptr) {
                q[u] = make_uint4(0u, 0u, 0u, 0u);
                e[u] = 0u;
                if (ok) {
                    q[u] = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(base) + from * c.D + l.o0);
                    e[u] = (isv ? c.vs : c.ks)[cache_scale(c, r.page, head, r.slot)];
                }
            } else {
                raw[u].load(base, from * c.D, l, ok);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int head = head0 + u * kAtOnce + sub;
            if (!l.in || head >= a.Hk) continue;
            const int64_t to = (row * a.Hk + head) * c.D;
            if (c.ks != nullptr) {
                const float unit = __uint_as_float(e[u] << 23);
                const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
                float f[16];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    e4m3_to_f(w[i] & 0xffffu, f[4 * i], f[4 * i + 1]);
                    e4m3_to_f(w[i] >> 16, f[4 * i + 2], f[4 * i + 3]);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] *= unit;
                Two<T>::store(out, to, l, f);
            } else {
                raw[u].a.store(static_cast<T *>(out) + to + l.o0);
                raw[u].b.store(static_cast<T *>(out) + to + l.o1);
            }
        }
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

// Whole vectors: the widths, all rows and all pointers allow 16 bytes at a time. (Norms of 2 x 8192 tokens, 40 heads of 128:
// 438 us a warp per row and channel by channel.)
bool vec_ok(const HeadArgs &a, bool f32, const void *const *ptrs, int n) {
    const int v = f32 ? 4 : 8;
    bool ok = a.D % 16 == 0 && a.R % 16 == 0 && a.q_stride % v == 0 && a.k_stride % v == 0 && a.v_stride % v == 0;
    for (int i = 0; i < n; ++i) ok = ok && aligned(ptrs[i], 16);
    return ok;
}

// How rows are shared out: `u` groups of heads to a warp, `tokens` tokens to a block.
struct VecPlan {
    int lpr, u, slices, tokens;
    unsigned blocks;
};
VecPlan vec_plan(const HeadArgs &a, int u, int blocks_per_sm) {
    VecPlan p;
    p.lpr = a.D <= 64 ? 4 : a.D <= 128 ? 8 : 16;
    const int at_once = 32 / p.lpr;
    auto slices = [&](int n) { return slices_of(a.Hq, n * at_once) + slices_of(a.Hk, n * at_once) + slices_of(a.Hv, n * at_once); };
    const int64_t most = (int64_t)sm_count() * blocks_per_sm;
    // few tokens: a warp for each group of heads
    p.u = u;
    if (ceil_div(a.seqs.rows, kVecWarps) * slices(u) < most) p.u = 1;
    p.slices = slices(p.u);
    // the tokens of a block: a multiple of its warps, so that `most` blocks or fewer cover all
    const int64_t chunks = most / p.slices < 1 ? 1 : most / p.slices;
    p.tokens = (int)(ceil_div(ceil_div(a.seqs.rows, chunks), kVecWarps) * kVecWarps);
    if (p.tokens < kVecWarps) p.tokens = kVecWarps;
    p.blocks = (unsigned)(ceil_div(a.seqs.rows, p.tokens) * p.slices);
    return p;
}

#define KDA_VEC_LAUNCH(kernel, T, U)                                                                                \
    switch (p.lpr) {                                                                                                \
        case 4: kernel<T, 4, U><<<p.blocks, 32 * kVecWarps, 0, stream>>>(a, p.slices, p.tokens); break;             \
        case 8: kernel<T, 8, U><<<p.blocks, 32 * kVecWarps, 0, stream>>>(a, p.slices, p.tokens); break;             \
        default: kernel<T, 16, U><<<p.blocks, 32 * kVecWarps, 0, stream>>>(a, p.slices, p.tokens); break;           \
    }
#define KDA_VEC(kernel, U)                                                                                          \
    if (f32) {                                                                                                      \
        if (p.u == 1) {                                                                                             \
            KDA_VEC_LAUNCH(kernel, float, 1)                                                                        \
        } else {                                                                                                    \
            KDA_VEC_LAUNCH(kernel, float, U / 2)                                                                    \
        }                                                                                                           \
    } else if (p.u == 1) {                                                                                          \
        KDA_VEC_LAUNCH(kernel, bf16, 1)                                                                             \
    } else {                                                                                                        \
        KDA_VEC_LAUNCH(kernel, bf16, U)                                                                             \
    }                                                                                                               \
    return cudaGetLastError();

cudaError_t launch_rows(const HeadArgs &a, bool f32, cudaStream_t stream) {
    if (sm_count() == 0) return cudaErrorInvalidDevice;
    const void *ptrs[] = {a.q, a.k, a.v, a.q_out, a.k_out};
    if (vec_ok(a, f32, ptrs, 5)) {
        const VecPlan p = vec_plan(a, f32 ? 2 : 4, 3);
        KDA_VEC(vec_rows_kernel, 4)
    }
    const unsigned blocks = any_blocks(a.seqs.rows * (a.Hq + a.Hk + a.Hv));
    if (f32)
        any_rows_kernel<float><<<blocks, 32 * kWarps, 0, stream>>>(a);
    else
        any_rows_kernel<bf16><<<blocks, 32 * kWarps, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_read(const HeadArgs &a, bool f32, cudaStream_t stream) {
    if (sm_count() == 0) return cudaErrorInvalidDevice;
    const void *ptrs[] = {a.q_out, a.k_out};
    if (vec_ok(a, f32, ptrs, 2)) {
        HeadArgs b = a;  // slices of keys, then of values
        b.Hv = b.Hk;
        const VecPlan p = vec_plan(b, f32 ? 2 : 4, 4);
        KDA_VEC(vec_read_kernel, 4)
    }
    const unsigned blocks = any_blocks(a.seqs.rows * 2 * a.Hk);
    if (f32)
        any_read_kernel<float><<<blocks, 32 * kWarps, 0, stream>>>(a);
    else
        any_read_kernel<bf16><<<blocks, 32 * kWarps, 0, stream>>>(a);
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
// The backward pass's arguments and blocks (as many rows of partial sums).
struct BwdPlan {
    HeadArgs a;
    bool vec;
    VecPlan p;
    unsigned blocks;
    size_t bytes;
};
BwdPlan bwd_plan(const kda_qk_norm_bwd_params &p, int64_t rows, unsigned int *err) {
    BwdPlan q;
    q.a = norm_args(p.f, rows, err);
    q.a.dq_out = p.dq_out;
    q.a.dk_out = p.dk_out;
    q.a.q_out = p.dq;
    q.a.k_out = p.dk;
    const bool f32 = p.f.dtype == KDA_DTYPE_F32;
    const void *ptrs[] = {p.f.q, p.f.k, p.dq_out, p.dk_out, p.dq, p.dk};
    q.vec = rows != 0 && vec_ok(q.a, f32, ptrs, 6);
    if (q.vec) {
        q.p = vec_plan(q.a, f32 ? 1 : 2, 2);
        q.blocks = q.p.blocks;
    } else {
        const int64_t most = (int64_t)sm_count() * 4, need = ceil_div(rows * (p.f.q_heads + p.f.k_heads), kWarps);
        q.blocks = (unsigned)(need < 1 ? 1 : need < most ? need : most);
    }
    q.bytes = p.dq_weight == nullptr && p.dk_weight == nullptr ? 0 : (size_t)q.blocks * 2 * p.f.D * sizeof(float);
    return q;
}

cudaError_t launch_bwd(const BwdPlan &q, bool f32, cudaStream_t stream) {
    const HeadArgs &a = q.a;
    if (sm_count() == 0) return cudaErrorInvalidDevice;
    if (q.vec) {
        const VecPlan &p = q.p;
        KDA_VEC(vec_rows_bwd_kernel, 2)
    }
    if (f32)
        any_rows_bwd_kernel<float><<<q.blocks, 32 * kWarps, 0, stream>>>(a);
    else
        any_rows_bwd_kernel<bf16><<<q.blocks, 32 * kWarps, 0, stream>>>(a);
    return cudaGetLastError();
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
    return status_of_cuda(launch_read(a, p->dtype == KDA_DTYPE_F32, stream));
}

size_t kda_qk_norm_bwd_workspace(const kda_qk_norm_bwd_params *p) {
    using namespace kda;
    int64_t rows = 0;
    if (p == nullptr || bwd_check(*p, &rows) != KDA_OK) return 0;
    return bwd_plan(*p, rows, nullptr).bytes;
}

int kda_qk_norm_bwd(const kda_qk_norm_bwd_params *p, cudaStream_t stream) {
    using namespace kda;
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    int64_t rows = 0;
    const int st = bwd_check(*p, &rows);
    if (st != KDA_OK) return st;
    BwdPlan q = bwd_plan(*p, rows, nullptr);
    if (p->workspace != nullptr && p->workspace_bytes < q.bytes) return KDA_ERR_INVALID_ARG;
    if (!aligned(p->workspace, 16)) return KDA_ERR_ALIGNMENT;
    if (rows == 0 && q.bytes == 0) return KDA_OK;
    cudaError_t e = device_error_word(&q.a.err);
    if (e != cudaSuccess) return status_of_cuda(e);
    Scratch ws;
    e = ws.get(p->workspace, q.bytes, stream);
    if (e != cudaSuccess) return status_of_cuda(e);
    q.a.partial = static_cast<float *>(ws.ptr);
    e = launch_bwd(q, p->f.dtype == KDA_DTYPE_F32, stream);
    const SumOuts outs{{p->dq_weight, p->dk_weight, nullptr, nullptr}, {p->f.D, p->f.D, 0, 0}};
    if (e == cudaSuccess && q.bytes != 0) e = launch_sum_partials(q.a.partial, q.blocks, 2 * (int64_t)p->f.D, outs, stream);
    return status_of_cuda(ws.release(e));
}

}  // extern "C"
