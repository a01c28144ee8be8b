// Rows of heads (kda_attention.h): the norms of queries and keys with the position rotation, their
// gradient, and the rows' way into the cache and out of it.
//
//   n = x r w, r = (mean x^2 + eps)^(-1/2);  pairs (a, b) of n -> (a cos - b sin, b cos + a sin)
//
// Gradient: g is dy with its pairs turned back, gw = g w, dx = r (gw - x r^2 mean(gw x)), dw = sum g x r.
#include <type_traits>

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
// LPR lanes share a row, 16 channels each as two chunks of 8; a warp holds a group of 32 / LPR rows (heads of one token) at
// a time. A block takes some tokens: first the place and the angles of each are worked out once and left in shared
// memory, then its warps go through the tokens' slices (a few groups of queries, keys or values), the
// next rows on their way while some are worked on. Arithmetic goes in pairs of fp32. The norms move 82 % of what a plain copy does
// (2 x 8192 tokens of 40 heads of 128, bf16: 60 us); what holds them is the instructions, about 240 for a group of 1 KB in
// and out (2.3 per clock and SM, waiting for shared memory, reciprocal roots and one another), with what belongs to a slice
// worked out once. The gradient (8191 tokens of 18 heads of 256: 49 us, 68 % of a copy) has 128 registers a thread,
// so only 16 warps on an SM. 8-bit writes: 38 us for 32761 tokens of 16 rows of 128, 77 %.
constexpr int kVecWarps = 8;
constexpr int kVecThreads = 32 * kVecWarps;
constexpr int kVecTokens = 32;  // of a block at a time, at most

struct VecArgs {
    HeadArgs h;
    int tokens;   // of a block at a time
    int batches;  // ceil(rows / tokens)
    int each;     // backward: groups of a slice, at most
};

// A token's place, in shared memory.
struct Place {
    int pos, page, slot;  // for the rotation; in the cache (page < 0: not there)
};

// What a block works out for its tokens `row0 ..` before their rows: places, cosines and sines. `count`: tokens that exist.
__device__ __forceinline__ void vec_places(const HeadArgs &a, int64_t row0, int count, Place *place) {
    // the sequence of the first token: how many offsets are not after it, counted by all threads at once
    int s0 = 0;
    if (a.seqs.cu != nullptr) {
        int n = 0;
        for (int i = threadIdx.x; i - (int)threadIdx.x < a.seqs.N; i += kVecThreads)  // the same number of turns for all
            n += __syncthreads_count(i < a.seqs.N && a.seqs.cu[i] <= row0);
        s0 = n < 1 ? 0 : n - 1;
    }
    if ((int)threadIdx.x >= count) return;
    const int64_t row = row0 + threadIdx.x;
    SeqAt at;
    if (a.seqs.cu == nullptr) {
        at = seq_find(a.seqs, row);
    } else {
        at.s = s0;
        while (at.s < a.seqs.N - 1 && a.seqs.cu[at.s + 1] <= row) ++at.s;
        seq_fill(a.seqs, row, at);
    }
    Place p;
    p.page = -1;
    p.slot = 0;
    p.pos = (int)(row - at.start);
    if (a.cached) {
        p.pos += cache_len(a.cache, at.s) - (int)(at.end - at.start);
        if (p.pos >= 0) p.page = cache_page(a.cache, at.s, p.pos, p.slot);
    }
    if (a.pos != nullptr) p.pos = a.pos[row];
    place[threadIdx.x] = p;
}
// `table`: of each token R / 2 cosines, sines and negative sines; the lane's two quads of each (pairs 8 j .. 8 j + 3 and the four
// after them) lie beside its neighbours': as they lie in the row, lanes would meet in the same banks.
__device__ __forceinline__ void vec_angles(const HeadArgs &a, int count, const Place *place, float *table) {
    const int half = a.R / 2;
    for (int i = threadIdx.x; i < count * half; i += kVecThreads) {
        const int t = i / half, e = i - t * half;
        float c, s;
        turn(a.freq[e], place[t].pos, c, s);
        float *to = table + t * 3 * half + ((e >> 2 & 1) * (half / 8) + (e >> 3)) * 4 + (e & 3);
        to[0] = c;
        to[half] = s;
        to[2 * half] = -s;
    }
}
// Where a block's share of all tokens begins.
__device__ __forceinline__ int64_t share_of(int64_t rows, int block) {
    const int64_t base = rows / gridDim.x, more = rows - base * gridDim.x;
    return block * base + (block < more ? block : more);
}
// The slices of heads of a token, `each` heads apiece.
__host__ __device__ __forceinline__ int slices_of(int heads, int each) { return (heads + each - 1) / each; }

// The lane's place in a row: two chunks of 8 channels, each beside its neighbours' (16 channels in one piece would leave every
// other 16 bytes to a second access).
struct LaneAt {
    int o0, o1;      // first channels of its two chunks
    bool in, turns;  // within the row; its channels are turned (pair e: 8 j + e)
};
__device__ __forceinline__ LaneAt lane_at(const HeadArgs &a, bool turned, int j) {
    LaneAt l;
    l.in = 16 * j < a.D;
    l.turns = turned && 16 * j < a.R;
    if (l.turns) {
        l.o0 = a.pairs ? 16 * j : 8 * j;
        l.o1 = a.pairs ? 16 * j + 8 : a.R / 2 + 8 * j;  // channels i and i + R / 2
    } else {
        const int from = turned ? a.R : 0;
        l.o0 = from / 2 + 8 * j;
        l.o1 = a.D / 2 + 8 * j;
    }
    return l;
}

// A warp's way through a block's (token, slice) items, every kVecWarps-th of them: the warps of a block read neighbouring rows
// at a time (a run of items for each warp, so that it has whole tokens, is slower: memory pages change more often).
struct Items {
    int token, slice, left;
    __device__ __forceinline__ Items(int warp, int tokens, int slices) {
        left = (tokens * slices - warp + kVecWarps - 1) / kVecWarps;
        token = warp / slices;
        slice = warp - token * slices;
    }
    __device__ __forceinline__ void step(int slices) {
        --left;
        slice += kVecWarps;
        while (slice >= slices) {
            slice -= slices;
            ++token;
        }
    }
};

// The two weights (ones where there is none), [2][4][LPR] quads: of lane j its first chunk's two and its second chunk's two.
template <int LPR>
__device__ __forceinline__ void vec_weights(const HeadArgs &a, float *w) {
    for (int i = threadIdx.x; i < 2 * 16 * LPR; i += kVecThreads) {
        const float *from = i < 16 * LPR ? a.qw : a.kw;
        const int k = i % (16 * LPR), quad = k / (4 * LPR), j = k / 4 % LPR;
        const LaneAt l = lane_at(a, true, j);
        w[i] = from != nullptr && l.in ? from[(quad < 2 ? l.o0 : l.o1 - 8) + 4 * quad + (k & 3)] : 1.f;
    }
}

template <typename T>
struct Two {
    Raw<T, 8> a, b;
    // of the row at `row`
    __device__ __forceinline__ void load(const T *row, const LaneAt &l, bool ok) {
        if (ok) {
            a.load(row + l.o0);
            b.load(row + l.o1);
        } else {
            a.zero();
            b.zero();
        }
    }
    __device__ __forceinline__ void unpack(f2 (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = a.pair(i);
            x[4 + i] = b.pair(i);
        }
    }
    static __device__ __forceinline__ void store(T *row, const LaneAt &l, const f2 (&x)[8]) {
        float t[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) upk(x[i], t[2 * i], t[2 * i + 1]);
        store_vec<T, 8>(row + l.o0, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) upk(x[4 + i], t[2 * i], t[2 * i + 1]);
        store_vec<T, 8>(row + l.o1, t);
    }
};
// Floats of shared memory as pairs, loaded where they are used (a copy in registers for all rows of a slice would cost a block
// on each SM).
__device__ __forceinline__ void lds4(f2 &x, f2 &y, uint32_t at) { asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(at)); }
// the lane's 16 weights
template <int LPR>
__device__ __forceinline__ void lds16(f2 (&x)[8], uint32_t at) {
#pragma unroll
    for (int i = 0; i < 4; ++i) lds4(x[2 * i], x[2 * i + 1], at + i * LPR * 16);
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The lane's 8 pairs by their angles: cosines, sines and negative sines of its pairs at shared addresses c, s, n, the second four
// `hop` bytes on.
__device__ __forceinline__ void turn_pairs(f2 (&x)[8], uint32_t c_at, uint32_t s_at, uint32_t n_at, int hop, bool pairs) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        f2 c[2], s[2], n[2];
        lds4(c[0], c[1], c_at + hop * h);
        lds4(s[0], s[1], s_at + hop * h);
        lds4(n[0], n[1], n_at + hop * h);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = 2 * h + k;
            if (pairs) {  // both numbers of a pair in one register
                float c0, c1, s0, s1, n0, n1, a, b;
                upk(c[k], c0, c1);
                upk(s[k], s0, s1);
                upk(n[k], n0, n1);
                upk(x[2 * i], a, b);
                x[2 * i] = fma2(pk(b, a), pk(n0, s0), mul2(x[2 * i], pk(c0, c0)));
                upk(x[2 * i + 1], a, b);
                x[2 * i + 1] = fma2(pk(b, a), pk(n1, s1), mul2(x[2 * i + 1], pk(c1, c1)));
            } else {
                const f2 a = x[i], b = x[4 + i];
                x[i] = fma2(b, n[k], mul2(a, c[k]));
                x[4 + i] = fma2(a, s[k], mul2(b, c[k]));
            }
        }
    }
}

// A row in 8 bits at `to`, its exponent byte at `scale`.
template <int LPR>
__device__ __forceinline__ void vec_put_e4m3(uint8_t *to, uint8_t *scale, const f2 (&x)[8], const LaneAt &l, bool ok, int j) {
    float top = 0.f;  // an infinity's exponent is 120 by the same rule; NaN is passed over
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float lo, hi;
        upk(x[i], lo, hi);
        top = fmaxf(top, fmaxf(fabsf(lo), fabsf(hi)));
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = row_exponent(top);
    const f2 unit = pk(pow2(-e), pow2(-e));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float f[4];
        upk(mul2(x[2 * i], unit), f[0], f[1]);
        upk(mul2(x[2 * i + 1], unit), f[2], f[3]);
        w[i] = e4m3_pair(f[0], f[1]) | e4m3_pair(f[2], f[3]) << 16;
    }
    if (!ok) return;
    *reinterpret_cast<uint2 *>(to + l.o0) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2 *>(to + l.o1) = make_uint2(w[2], w[3]);
    if (j == 0) *scale = (uint8_t)(e + 127);
}

// Queries and keys normed and turned (kNorm), that with keys and values into the cache (kStep), or the latter alone (kWrite).
enum Mode { kNorm, kStep, kWrite };

template <typename T, int LPR, int U, int MODE>
__global__ void __launch_bounds__(kVecThreads, MODE == kWrite ? 4 : 3) vec_rows_kernel(const __grid_constant__ VecArgs v) {
    constexpr int kAtOnce = 32 / LPR;
    __shared__ Place place[kVecTokens];
    extern __shared__ __align__(16) float mem[];
    const HeadArgs &a = v.h;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / LPR, j = lane % LPR;
    if (blockIdx.x == 0) seq_check(a.seqs, a.err, threadIdx.x, kVecThreads);
    float *weights = mem, *table = mem + 32 * LPR;
    constexpr int per = U * kAtOnce;  // heads of a slice
    const int hop = kAtOnce * a.D;    // channels between groups
    const int nq = slices_of(a.Hq, per), nk = slices_of(a.Hk, per), slices = nq + nk + slices_of(a.Hv, per);
    const LaneAt lt = lane_at(a, true, j), lv = lane_at(a, false, j);
    const float inv_d = 1.f / (float)a.D;
    if constexpr (MODE != kWrite) vec_weights<LPR>(a, weights);

    // the block's tokens, v.tokens at a time
    const int64_t end = share_of(a.seqs.rows, blockIdx.x + 1);
#pragma unroll 1
    for (int64_t row0 = share_of(a.seqs.rows, blockIdx.x); row0 < end; row0 += v.tokens) {
        const int count = end - row0 < v.tokens ? (int)(end - row0) : v.tokens;
        Items it(warp, count, slices);
        // of the slice ahead: queries, keys or values (0, 1, 2), the lane's first head, heads from there on, and its row
        int part = 0, head = 0, left = 0;
        const T *in = nullptr;
        auto aim = [&] {
            part = it.slice < nq ? 0 : it.slice < nq + nk ? 1 : 2;
            const int first = (it.slice - (part == 0 ? 0 : part == 1 ? nq : nq + nk)) * per;
            const int heads = part == 0 ? a.Hq : part == 1 ? a.Hk : a.Hv;
            head = first + sub;
            left = it.left > 0 ? (first + per < heads ? first + per : heads) - head : 0;
            in = static_cast<const T *>(part == 0 ? a.q : part == 1 ? a.k : a.v) +
                 (row0 + it.token) * (part == 0 ? a.q_stride : part == 1 ? a.k_stride : a.v_stride) + (int64_t)head * a.D;
        };
        Two<T> raw[U];
        aim();
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u].load(in + u * hop, part == 2 ? lv : lt, left > u * kAtOnce && lt.in);
        __syncthreads();  // the places and angles of the tokens before are done with
        vec_places(a, row0, count, place);
        __syncthreads();
        if (MODE != kWrite && a.R > 0) {
            vec_angles(a, count, place, table);
            __syncthreads();
        }
#pragma unroll 1
        while (it.left > 0) {
            const bool isq = part == 0, isv = part == 2, turns = MODE != kWrite && !isv && lt.turns;
            const LaneAt l = isv ? lv : lt;
            const bool normed = MODE != kWrite && !isv && (isq ? a.qw : a.kw) != nullptr;
            T *out = static_cast<T *>(isq ? a.q_out : a.k_out);
            const bool to_out = MODE != kWrite && !isv && out != nullptr;
            if constexpr (MODE != kWrite) out += ((row0 + it.token) * (isq ? a.Hq : a.Hk) + head) * a.D;
            const uint32_t wt_at = smem_u32(weights) + (isq ? 0 : 64 * LPR) + 16 * j;
            const uint32_t angles = smem_u32(table) + 4 * (it.token * (a.R / 2) * 3 + 4 * j);
            // the row's place in the cache
            bool put = false;
            uint8_t *to = nullptr, *scale = nullptr;
            if constexpr (MODE != kNorm) {
                const Place p = place[it.token];
                if (!isq && p.page >= 0) {
                    put = true;
                    to = static_cast<uint8_t *>(isv ? a.cache.v : a.cache.k) +
                         cache_row(a.cache, p.page, head, p.slot) * a.D * (a.cache.ks != nullptr ? 1 : (int)sizeof(T));
                    scale = (isv ? a.cache.vs : a.cache.ks) + cache_scale(a.cache, p.page, head, p.slot);
                }
            }
            const int live = lt.in ? left : 0;
            it.step(slices);
            aim();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool ok = live > u * kAtOnce;
                f2 x[8];
                raw[u].unpack(x);
                raw[u].load(in + u * hop, part == 2 ? lv : lt, lt.in && left > u * kAtOnce);
                if (normed) {
                    f2 q = mul2(x[0], x[0]);
#pragma unroll
                    for (int i = 1; i < 8; ++i) q = fma2(x[i], x[i], q);
                    const float inv = rsqrtf(row_sum<LPR>(hsum2(q)) * inv_d + a.eps);
                    const f2 by = pk(inv, inv);
                    if (lt.in) {
                        f2 wt[8];
                        lds16<LPR>(wt, wt_at);
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = mul2(x[i], mul2(wt[i], by));
                    }
                }
                if (turns) turn_pairs(x, angles, angles + 2 * a.R, angles + 4 * a.R, a.R, a.pairs);
                if (to_out && ok) Two<T>::store(out + u * hop, l, x);
                if (MODE != kNorm && put) {
                    const int64_t at = (int64_t)u * hop * a.cache.page;
                    if (a.cache.ks != nullptr)
                        vec_put_e4m3<LPR>(to + at, scale + u * kAtOnce * a.cache.page, x, l, ok, j);
                    else if (ok)
                        Two<T>::store(reinterpret_cast<T *>(to) + at, l, x);
                }
            }
        }
    }
}

// The gradient: blocks go through batches of tokens, each lane adds up the weights' gradients at its channels.
template <typename T, int LPR>
__global__ void __launch_bounds__(kVecThreads, 2) vec_rows_bwd_kernel(const __grid_constant__ VecArgs v) {
    constexpr int kAtOnce = 32 / LPR;
    __shared__ Place place[kVecTokens];
    extern __shared__ __align__(16) float mem[];
    const HeadArgs &a = v.h;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / LPR, j = lane % LPR;
    if (blockIdx.x == 0) seq_check(a.seqs, a.err, threadIdx.x, kVecThreads);
    // shared floats: weights, the lanes' sums of the weights' gradients ([2][4] of four channels, a thread's 16 bytes beside its
    // neighbours'), angles (at the end a row of sums for each warp)
    float *weights = mem, *table = mem + 32 * LPR + 32 * kVecThreads;
    float4 *sums = reinterpret_cast<float4 *>(mem + 32 * LPR) + threadIdx.x;
    const LaneAt l = lane_at(a, true, j);
    const int per = v.each * kAtOnce, hop = kAtOnce * a.D;
    const int nq = slices_of(a.Hq, per), slices = nq + slices_of(a.Hk, per);
    const float inv_d = 1.f / (float)a.D;
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[i * kVecThreads] = make_float4(0.f, 0.f, 0.f, 0.f);
    vec_weights<LPR>(a, weights);

#pragma unroll 1
    for (int batch = blockIdx.x; batch < v.batches; batch += gridDim.x) {
        const int64_t row0 = (int64_t)batch * v.tokens;
        const int count = a.seqs.rows - row0 < v.tokens ? (int)(a.seqs.rows - row0) : v.tokens;
        Items it(warp, count, slices);
        Two<T> raw, raw_g;
        bool isq = true;
        int left = 0;
        int64_t dense = 0;
        const T *in = nullptr, *dout = nullptr;
        auto aim = [&] {
            isq = it.slice < nq;
            const int first = (isq ? it.slice : it.slice - nq) * per, heads = isq ? a.Hq : a.Hk, head = first + sub;
            left = it.left > 0 ? (first + per < heads ? first + per : heads) - head : 0;
            dense = ((row0 + it.token) * heads + head) * a.D;
            dout = static_cast<const T *>(isq ? a.dq_out : a.dk_out) + dense;
            in = static_cast<const T *>(isq ? a.q : a.k) + (row0 + it.token) * (isq ? a.q_stride : a.k_stride) + (int64_t)head * a.D;
        };
        auto fetch = [&](bool ok) {
            raw_g.load(dout, l, ok);
            raw.load(in, l, ok && (isq ? a.qw : a.kw) != nullptr);
        };
        aim();
        fetch(left > 0 && l.in);
        if (a.R > 0) vec_places(a, row0, count, place);
        __syncthreads();
        if (a.R > 0) {
            vec_angles(a, count, place, table);
            __syncthreads();
        }
#pragma unroll 1
        while (it.left > 0) {
            const bool normed = (isq ? a.qw : a.kw) != nullptr;
            T *out = static_cast<T *>(isq ? a.q_out : a.k_out) + dense;
            const uint32_t wt_at = smem_u32(weights) + (isq ? 0 : 64 * LPR) + 16 * j;
            const uint32_t angles = smem_u32(table) + 4 * (it.token * (a.R / 2) * 3 + 4 * j);
            float4 *to = sums + (isq ? 0 : 4) * kVecThreads;
            f2 total[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) total[i] = pk(0.f, 0.f);
            int now_left = left, n = v.each;
            bool last;
#pragma unroll 1
            do {
                const bool there = now_left > 0, ok = there && l.in;
                f2 g[8], x[8];
                raw_g.unpack(g);
                raw.unpack(x);
                now_left -= kAtOnce;
                last = --n == 0 || __all_sync(0xffffffffu, now_left <= 0);
                if (last) {
                    it.step(slices);
                    aim();
                } else {
                    in += hop;
                    dout += hop;
                }
                fetch((last ? left : now_left) > 0 && l.in);
                if (l.turns) turn_pairs(g, angles, angles + 4 * a.R, angles + 2 * a.R, a.R, a.pairs);  // back
                if (normed) {
                    f2 wt[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) wt[i] = pk(0.f, 0.f);
                    if (l.in) lds16<LPR>(wt, wt_at);
                    f2 q = mul2(x[0], x[0]), m = pk(0.f, 0.f);
#pragma unroll
                    for (int i = 1; i < 8; ++i) q = fma2(x[i], x[i], q);
                    // a row of the last group that is not there adds zeros to the weights' gradients, with eps = 0 too
                    const float mean = row_sum<LPR>(hsum2(q)) * inv_d;
                    const float inv = there ? rsqrtf(mean + a.eps) : 0.f;
                    const f2 by = pk(inv, inv);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const f2 gx = mul2(g[i], x[i]);
                        m = fma2(gx, wt[i], m);
                        total[i] = fma2(gx, by, total[i]);
                        g[i] = mul2(g[i], mul2(wt[i], by));
                    }
                    const float k = row_sum<LPR>(hsum2(m)) * inv_d * inv * inv * inv;
#pragma unroll
                    for (int i = 0; i < 8; ++i) g[i] = fma2(x[i], pk(-k, -k), g[i]);
                }
                if (ok) Two<T>::store(out, l, g);
                out += hop;
            } while (!last);
            if (normed) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 old = to[i * kVecThreads];
                    float t[4];
                    upk(total[2 * i], t[0], t[1]);
                    upk(total[2 * i + 1], t[2], t[3]);
                    to[i * kVecThreads] = make_float4(old.x + t[0], old.y + t[1], old.z + t[2], old.w + t[3]);
                }
            }
        }
        __syncthreads();  // the angles of the next batch go where these are
    }
    if (a.partial == nullptr) return;
    // over the rows of a warp, then the block's warps in order
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            const float4 t4 = sums[(4 * part + i) * kVecThreads];
            float t[4] = {t4.x, t4.y, t4.z, t4.w};
#pragma unroll
            for (int h = 0; h < 4; ++h) {
#pragma unroll
                for (int o = LPR; o < 32; o <<= 1) t[h] += __shfl_xor_sync(0xffffffffu, t[h], o);
                if (sub == 0 && l.in) table[warp * a.D + (i < 2 ? l.o0 : l.o1 - 8) + 4 * i + h] = t[h];
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < a.D; i += kVecThreads) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < kVecWarps; ++w) t += table[w * a.D + i];
            a.partial[((int64_t)blockIdx.x * 2 + part) * a.D + i] = t;
        }
        __syncthreads();
    }
}

// Rows of the cache into contiguous ones: a lane has 16 channels of a row, and U rows on their way at a time. A block takes
// some tokens; their rows in the order (token, keys or values, head).
template <typename T, int LPR, int U, int SCALED>
__global__ void __launch_bounds__(kVecThreads, SCALED ? 4 : 3) vec_read_kernel(const __grid_constant__ VecArgs v) {
    constexpr int kAtOnce = 32 / LPR;
    __shared__ Place place[kVecThreads];
    const HeadArgs &a = v.h;
    const Cache &c = a.cache;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / LPR, j = lane % LPR;
    if (blockIdx.x == 0) seq_check(a.seqs, a.err, threadIdx.x, kVecThreads);
    const int64_t row0 = (int64_t)blockIdx.x * v.tokens;
    const int count = a.seqs.rows - row0 < v.tokens ? (int)(a.seqs.rows - row0) : v.tokens;
    vec_places(a, row0, count, place);
    __syncthreads();
    const LaneAt l = lane_at(a, false, j);
    const int each = 2 * a.Hk, all = count * each;
#pragma unroll 1
    for (int first = warp * U * kAtOnce; first < all; first += kVecWarps * U * kAtOnce) {
        uint4 q[SCALED ? U : 1];
        uint32_t e[SCALED ? U : 1];
        Two<T> raw[SCALED ? 1 : U];
        // row `first + sub` and those kAtOnce further on: head h of the token's keys and values
        int token = (first + sub) / each, h = first + sub - token * each;
        const int token0 = token, h0 = h;
        auto next = [&] {
            h += kAtOnce;
            while (h >= each) {
                h -= each;
                ++token;
            }
        };
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool isv = h >= a.Hk;
            Place p{0, -1, 0};
            if (token < count) p = place[token];
            const bool ok = l.in && p.page >= 0;
            const int head = isv ? h - a.Hk : h;
            const int64_t from = ok ? cache_row(c, p.page, head, p.slot) : 0;
            const void *base = isv ? c.v : c.k;
            if constexpr (SCALED) {
                q[u] = make_uint4(0u, 0u, 0u, 0u);
                e[u] = 0u;
                if (ok) {
                    const uint8_t *row = static_cast<const uint8_t *>(base) + from * c.D;
                    const uint2 lo = *reinterpret_cast<const uint2 *>(row + l.o0), hi = *reinterpret_cast<const uint2 *>(row + l.o1);
                    q[u] = make_uint4(lo.x, lo.y, hi.x, hi.y);
                    e[u] = (isv ? c.vs : c.ks)[cache_scale(c, p.page, head, p.slot)];
                }
            } else {
                raw[u].load(static_cast<const T *>(base) + from * c.D, l, ok);
            }
            next();
        }
        token = token0;
        h = h0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (l.in && token < count) {
                const bool isv = h >= a.Hk;
                T *out = static_cast<T *>(isv ? a.q_out : a.k_out) + ((row0 + token) * a.Hk + (isv ? h - a.Hk : h)) * c.D;
                if constexpr (SCALED) {
                    // a scale of 2^-127 (byte 0), which no row written here has, is below fp32's normal numbers: 0
                    const f2 unit = pk(__uint_as_float(e[u] << 23), __uint_as_float(e[u] << 23));
                    const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
                    f2 x[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float f[4];
                        e4m3_to_f(w[k] & 0xffffu, f[0], f[1]);
                        e4m3_to_f(w[k] >> 16, f[2], f[3]);
                        x[2 * k] = mul2(pk(f[0], f[1]), unit);
                        x[2 * k + 1] = mul2(pk(f[2], f[3]), unit);
                    }
                    Two<T>::store(out, l, x);
                } else {
                    raw[u].a.store(out + l.o0);
                    raw[u].b.store(out + l.o1);
                }
            }
            next();
        }
    }
}

// ---- host side -------------------------------------------------------------------------------
int elem_size(int dtype) { return dtype == KDA_DTYPE_BF16 ? 2 : 4; }

int sizes_check(int B, int T, const int32_t *cu, int dtype, int64_t heads, int64_t *rows) {
    if (B < 1 || T < 0 || heads < 1) return KDA_ERR_INVALID_ARG;
    if (dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_F32) return KDA_ERR_UNSUPPORTED;
    *rows = cu != nullptr ? T : (int64_t)B * T;
    // counts of heads of tokens go a block's stride beyond their number
    if (*rows != 0 && heads > (INT32_MAX - (1 << 16)) / *rows) return KDA_ERR_UNSUPPORTED;
    return aligned(cu, 4) ? KDA_OK : KDA_ERR_ALIGNMENT;
}
int stride_check(int64_t given, int64_t dense) { return given != 0 && given < dense ? KDA_ERR_INVALID_ARG : KDA_OK; }

// Which outputs a call writes: q_out and k_out (the forward pass), k_out only if it is given (single tokens), or neither (gradient).
enum Outs { kBoth, kKeysIfGiven, kNeither };

int norm_check(const kda_qk_norm_params &p, Outs outs, int64_t *rows) {
    const bool q_out = outs != kNeither, k_out = outs == kBoth || (outs == kKeysIfGiven && p.k_out != nullptr);
    if (p.q_heads < 1 || p.k_heads < 1 || p.D < 1 || p.R < 0 || p.R % 2 != 0 || p.R > p.D || !(p.eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    const int st = sizes_check(p.B, p.T, p.cu_seqlens, p.dtype, p.q_heads + 2 * (int64_t)p.k_heads, rows);
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
// 60 us, and 439 a warp per row and channel by channel; gradient of 8191 tokens 49 and 292, 8-bit writes 38 and 324.)
bool vec_ok(const HeadArgs &a, bool f32, const void *const *ptrs, int n) {
    const int v = f32 ? 4 : 8;
    bool ok = a.D % 16 == 0 && a.R % 16 == 0 && a.q_stride % v == 0 && a.k_stride % v == 0 && a.v_stride % v == 0;
    for (int i = 0; i < n; ++i) ok = ok && aligned(ptrs[i], 16);
    return ok;
}

// How tokens are shared out.
struct VecPlan {
    VecArgs v;
    int lpr, u;
    unsigned blocks;
    size_t smem;
};
VecPlan vec_plan(const HeadArgs &a, bool f32) {
    VecPlan p;
    p.v.h = a;
    p.lpr = a.D <= 64 ? 4 : a.D <= 128 ? 8 : 16;
    // 8-bit writes with 8, 16 and 32 tokens: 20000 tokens of 8 heads 27, 27 and 31 us (the last blocks run alone), 32761 40, 39 and 38,
    // 65536 76, 69 and 70, 32761 of 2 heads 33, 29 and 27. Norms alike from 9 to 16.
    p.v.tokens = a.q != nullptr ? 12 : 16;
    p.v.each = 4;  // gradient: groups of a slice (8191 tokens of 18 heads of 256: 49 us with two or four, 63 with eight, which 18 heads do not fill)
    p.u = f32 ? 1 : 2;  // groups of a warp on their way: 16 registers each (bf16 norms of 2 x 8192 tokens 60 us with two, 62 with one; 8-bit writes 38, 42)
    // few tokens: a warp for each group of heads, and as few tokens in a block as keep its warps busy (8 single tokens into the
    // cache: 4.4 us, and 11 with twelve tokens in a block)
    const int64_t sms = sm_count();
    if (a.seqs.rows < 4 * sms * p.v.tokens) {
        const int groups = slices_of(a.Hq + a.Hk + a.Hv, 32 / p.lpr);
        p.v.tokens = groups >= kVecWarps ? 1 : kVecWarps / groups;
        while (p.v.tokens < 16 && ceil_div(a.seqs.rows, p.v.tokens) > 4 * sms) p.v.tokens *= 2;
        if (a.seqs.rows * groups < 4 * sms * kVecWarps * 4) p.v.each = p.u = 1;
    }
    p.v.batches = (int)ceil_div(a.seqs.rows, p.v.tokens);
    // With norms and angles, blocks that stay and go through shares of all tokens (bf16 norms of 2 x 4096 tokens of 40 heads of 128 33 us, and 35
    // with a block for each 12 tokens; 2 x 8192 60 both ways; 2 x 30000 of 10 heads 88 and 90), but not in fp32 (2 x 8192 tokens 121 us,
    // and 111 with a block for each 12; 2 x 30000 of 10 heads 102 and 104); rows that are only written, 16 tokens a block (38 us, and 40 with blocks that stay).
    p.blocks = (unsigned)(a.q == nullptr || f32 || p.v.batches < 3 * sms ? p.v.batches : 3 * sms);
    p.smem = ((size_t)p.v.tokens * (a.R / 2) * 3 + 32 * p.lpr) * sizeof(float);  // at most 26 KB
    return p;
}

template <int N>
using Int = std::integral_constant<int, N>;
// Calls f with the lanes of a row as a constant.
template <typename F>
cudaError_t with_lpr(const VecPlan &p, F f) {
    if (p.lpr == 4)
        f(Int<4>{});
    else if (p.lpr == 8)
        f(Int<8>{});
    else
        f(Int<16>{});
    return cudaGetLastError();
}
template <typename T, int U, int MODE>
cudaError_t vec_mode(const VecPlan &p, cudaStream_t stream) {
    return with_lpr(p, [&](auto lpr) { vec_rows_kernel<T, decltype(lpr)::value, U, MODE><<<p.blocks, kVecThreads, p.smem, stream>>>(p.v); });
}
template <typename T, int MODE>
cudaError_t vec_groups(const VecPlan &p, cudaStream_t stream) {
    if constexpr (sizeof(T) == 2)  // fp32 has one on its way
        if (p.u == 2) return vec_mode<T, 2, MODE>(p, stream);
    return vec_mode<T, 1, MODE>(p, stream);
}
template <typename T>
cudaError_t vec_rows(const VecPlan &p, cudaStream_t stream) {
    if (!p.v.h.cached) return vec_groups<T, kNorm>(p, stream);
    return p.v.h.q != nullptr ? vec_groups<T, kStep>(p, stream) : vec_groups<T, kWrite>(p, stream);
}
template <typename T>
cudaError_t vec_bwd(const VecPlan &p, cudaStream_t stream) {
    return with_lpr(p, [&](auto lpr) { vec_rows_bwd_kernel<T, decltype(lpr)::value><<<p.blocks, kVecThreads, p.smem, stream>>>(p.v); });
}
// MOST: rows of a lane on their way where there are enough
template <typename T, int MOST, int SCALED>
cudaError_t vec_read(const VecPlan &p, cudaStream_t stream) {
    auto rows = [&](auto u) {
        return with_lpr(p, [&](auto lpr) {
            vec_read_kernel<T, decltype(lpr)::value, decltype(u)::value, SCALED><<<p.blocks, kVecThreads, p.smem, stream>>>(p.v);
        });
    };
    return p.u == 1 ? rows(Int<1>{}) : rows(Int<MOST>{});
}

cudaError_t launch_rows(const HeadArgs &a, bool f32, cudaStream_t stream) {
    if (sm_count() == 0) return cudaErrorInvalidDevice;
    const void *ptrs[] = {a.q, a.k, a.v, a.q_out, a.k_out};
    if (vec_ok(a, f32, ptrs, 5)) {
        const VecPlan p = vec_plan(a, f32);
        return f32 ? vec_rows<float>(p, stream) : vec_rows<bf16>(p, stream);
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
        VecPlan p = vec_plan(a, f32);
        // As many tokens in a block as its warps have rows on their way: eight of a lane, four in the data's type, two in fp32 (8-bit to
        // bf16, 32768 tokens of 8 heads of 128: 38 us with eight, 43 with four; to fp32 71 with two, 76 with four), or one where there
        // would not be two blocks for each SM (800 tokens: 3.0 us, and 5.9).
        const bool scaled = a.cache.ks != nullptr;
        const int64_t sms = sm_count();
        auto tokens = [&](int u) {
            const int n = kVecWarps * u * 32 / p.lpr / (2 * a.Hk);
            return n < 1 ? 1 : n > kVecThreads ? kVecThreads : n;
        };
        p.u = f32 ? 2 : scaled ? 8 : 4;
        if (ceil_div(a.seqs.rows, tokens(p.u)) < 2 * sms) p.u = 1;
        p.v.tokens = tokens(p.u);
        p.v.batches = (int)ceil_div(a.seqs.rows, p.v.tokens);
        p.blocks = (unsigned)p.v.batches;
        p.smem = 0;
        if (f32) return scaled ? vec_read<float, 2, 1>(p, stream) : vec_read<float, 2, 0>(p, stream);
        return scaled ? vec_read<bf16, 8, 1>(p, stream) : vec_read<bf16, 4, 0>(p, stream);
    }
    const unsigned blocks = any_blocks(a.seqs.rows * 2 * a.Hk);
    if (f32)
        any_read_kernel<float><<<blocks, 32 * kWarps, 0, stream>>>(a);
    else
        any_read_kernel<bf16><<<blocks, 32 * kWarps, 0, stream>>>(a);
    return cudaGetLastError();
}

int bwd_check(const kda_qk_norm_bwd_params &p, int64_t *rows) {
    const int st = norm_check(p.f, kNeither, rows);
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
        q.p = vec_plan(q.a, f32);
        q.p.blocks = (unsigned)q.p.v.batches;
        const int sms = sm_count();  // 0 without a device: the call itself reports that
        const unsigned most = sms > 0 ? 2 * sms : 1;
        // at most as many tokens at a time as there is room for the angles of (46 KB in all)
        int cap = (46 * 1024 / 4 - 32 * q.p.lpr - 32 * kVecThreads) / (p.f.R / 2 * 3 + 1);
        cap = cap > kVecTokens ? kVecTokens : cap;
        if (q.p.blocks > most || q.p.v.tokens > cap) {
            const int64_t times = ceil_div(rows, (int64_t)most * cap);  // the same for every block
            q.p.v.tokens = (int)ceil_div(rows, most * times);
            q.p.v.batches = (int)ceil_div(rows, q.p.v.tokens);
            q.p.blocks = q.p.v.batches < (int)most ? (unsigned)q.p.v.batches : most;
        }
        q.blocks = q.p.blocks;
        const int table = q.p.v.tokens * (p.f.R / 2) * 3;
        q.p.smem = (size_t)(32 * q.p.lpr + 32 * kVecThreads + (table > kVecWarps * p.f.D ? table : kVecWarps * p.f.D)) * sizeof(float);
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
        VecPlan p = q.p;
        p.v.h = a;
        return f32 ? vec_bwd<float>(p, stream) : vec_bwd<bf16>(p, stream);
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
    const int st = norm_check(*p, kBoth, &rows);
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
    int st = norm_check(p->f, kKeysIfGiven, &rows);
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
    int st = sizes_check(p->B, p->T, p->cu_seqlens, p->dtype, 2 * (int64_t)p->cache.heads, &rows);
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
    int st = sizes_check(p->B, p->T, p->cu_seqlens, p->dtype, 2 * (int64_t)p->cache.heads, &rows);
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
