// What the kernels of the selective scan share: arguments, step sizes and decays, states in memory, and
// the carry between chunks.
//
// Two layouts. The walks (forward, and the gradient's local pass): a thread owns up to 16 states of one or two
// channels, 17 to 64 states take 2 or 4 lanes. The step and the gradient's third kernel: four neighbouring lanes
// share channels, lane nl holding states nl NP .. nl NP + NP - 1 (NP = 2, 4, 8, 16: the smallest that
// holds N; the rest are zero states that stay zero).
#pragma once

#include "mixer_common.cuh"

namespace kda {
namespace scan {

using namespace mix;

constexpr int kDB = 64;  // channels per block of the gradient's third kernel
constexpr int kLN = 4;   // lanes that share a channel in the second layout
constexpr int kMaxN = 64;

struct ScanArgs {
    const void *u, *dt;
    const float *A;
    const void *B, *C;
    const float *D;
    const void *z;
    const float *bias, *h0;
    void *y;
    float *ht;
    int64_t us, dts, bs, cs, zs;  // elements between tokens
    int ch, N, G, chg;            // channels, states, groups, channels per group
    int blocks_per_group;
    int softplus;
    int vec;                      // channels may be read several at a time (each file's kernels say how many)
    int vec_states;               // A, h0, ht: 16 bytes at a time
    Seqs seqs;
    int64_t chunk;                // rows per chunk (all sequences' rows together); 0: one block per sequence
    int64_t nchunks;
    float *hchunk;                // [nchunks][ch][N]: a chunk's end state, then the state it starts from
    float *schunk;                // [nchunks][ch]: sum of the step sizes in a chunk
    unsigned int *err;
};

inline int np_of(int N) { return N <= 8 ? 2 : (N <= 16 ? 4 : (N <= 32 ? 8 : 16)); }

// A block's channels (gradient's third kernel): group g, the first channel, and how many of the 64 exist.
struct Chans {
    int g, d0, n;
};
__device__ __forceinline__ Chans chans_of(const ScanArgs &a, int block) {
    Chans c;
    c.g = block / a.blocks_per_group;
    const int first = (block % a.blocks_per_group) * kDB;
    c.d0 = c.g * a.chg + first;
    c.n = a.chg - first < kDB ? a.chg - first : kDB;
    return c;
}

// 8 channels of one token, zeros where there are none
template <typename T>
__device__ __forceinline__ void load8(Raw<T, 8> &r, const void *base, int64_t at, int n, bool vec) {
    const T *p = static_cast<const T *>(base) + at;
    if (vec && n >= 8)
        r.load(p);
    else if (n > 0)
        r.load_some(p, n);
    else
        r.zero();
}
template <typename T>
__device__ __forceinline__ void store8(void *base, int64_t at, const float (&f)[8], int n, bool vec) {
    Raw<T, 8> r;
    r.pack(f);
    T *p = static_cast<T *>(base) + at;
    if (vec && n >= 8)
        r.store(p);
    else if (n > 0)
        r.store_some(p, n);
}

// Step size from dt + dt_bias. In fp32 by CUDA's log1pf and expf; for bf16 inputs, whose own rounding is
// half a step (2^-8), on the special-function unit and a polynomial: relative error under 1e-6, below -10 up
// to 8e-8 |s| more (the exponent s log2 e is rounded once).
template <typename T>
__device__ __forceinline__ float step_of(float s, bool softplus) {
    if (!softplus) return s;
    if constexpr (sizeof(T) == 4)
        return softplus_f(s);
    else
        return tcu::softplus_fast(s);
}

// Decays exp(delta A) of a pair, A2 = A log2 e. The special-function unit's 2^x comes out low by 2e-8 on
// average over the exponents that matter for a long memory (-1/2 to -1/256, measured), which a state that
// remembers hundreds of steps adds up; kExpFix in the exponent (2e-8 log2 e, free in the multiply-add)
// centres it. With delta = 0 the result is still exactly 1.
constexpr float kExpFix = 3e-8f;
__device__ __forceinline__ f2 decay2(f2 delta, f2 A2) { return exp2_2(fma2(delta, A2, pk(kExpFix, kExpFix))); }

// Four values of each lane, added over the kLN lanes that share channels: lane nl returns the total of
// value nl. Three exchanges instead of the eight of four butterflies.
__device__ __forceinline__ float sum_lanes(const float (&p)[4], int nl) {
    const bool hi = nl & 2, odd = nl & 1;
    const float a0 = hi ? p[0] : p[2], a1 = hi ? p[1] : p[3];
    float b0 = hi ? p[2] : p[0], b1 = hi ? p[3] : p[1];
    b0 += __shfl_xor_sync(0xffffffffu, a0, 2);
    b1 += __shfl_xor_sync(0xffffffffu, a1, 2);
    const float s = odd ? b0 : b1, k = odd ? b1 : b0;
    return k + __shfl_xor_sync(0xffffffffu, s, 1);
}

// The states of channel d at `at` (of [..][ch][N]) for this lane, zeros past N and for no channel.
template <int NP>
__device__ __forceinline__ void load_states(float (&h)[NP], const float *base, int64_t at, int nl, int N, bool live) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int n = nl * NP + i;
        h[i] = live && n < N ? base[at + n] : 0.f;
    }
}
template <int NP>
__device__ __forceinline__ void store_states(const float (&h)[NP], float *base, int64_t at, int nl, int N, bool live) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int n = nl * NP + i;
        if (live && n < N) base[at + n] = h[i];
    }
}
// A thread's NS states of a channel, at `at` = first state of [..][N], zeros past N.
template <int NS>
__device__ __forceinline__ void get_states(f2 (&h)[NS / 2], const float *base, int64_t at, int n0, int N, bool live, bool vec) {
    if (live && vec) {
#pragma unroll
        for (int i = 0; i < NS / 4; ++i) {
            const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(base + at + n0 + 4 * i);
            h[2 * i] = q.x;
            h[2 * i + 1] = q.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NS / 2; ++i) {
            const int n = n0 + 2 * i;
            h[i] = pk(live && n < N ? base[at + n] : 0.f, live && n + 1 < N ? base[at + n + 1] : 0.f);
        }
    }
}
template <int NS>
__device__ __forceinline__ void put_states(const f2 (&h)[NS / 2], float *base, int64_t at, int n0, int N, bool live, bool vec) {
    if (!live) return;
    if (vec) {
#pragma unroll
        for (int i = 0; i < NS / 4; ++i)
            *reinterpret_cast<ulonglong2 *>(base + at + n0 + 4 * i) = make_ulonglong2(h[2 * i], h[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < NS / 2; ++i) {
            const int n = n0 + 2 * i;
            float lo, hi;
            upk(h[i], lo, hi);
            if (n < N) base[at + n] = lo;
            if (n + 1 < N) base[at + n + 1] = hi;
        }
    }
}

// Chunk end states to chunk start states, in place; one thread per (channel, state) walks
// the chunks, 16 loads ahead, in blocks of 256. A chunk in which a sequence starts does not pass its start
// state on. Chunk 0 starts a sequence: its own start state is not read.
__device__ __forceinline__ void carry_states(const ScanArgs &a) {
    constexpr int kAhead = 16;
    __shared__ bool starts[256];  // whether a sequence starts in a chunk, 256 chunks at a time
    const int64_t total = (int64_t)a.ch * a.N;
    const int64_t at_e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t e = at_e < total ? at_e : total - 1;  // the block's barriers want every thread
    const int d = (int)(e / a.N);
    const float A = a.A[e] * kLog2e;
    float in = 0.f;
    for (int64_t cb = 0; cb < a.nchunks; cb += kAhead) {
        if (cb % 256 == 0) {
            __syncthreads();
            const int64_t c0 = (cb + threadIdx.x) * a.chunk, c1 = c0 + a.chunk;
            starts[threadIdx.x] = c1 <= a.seqs.rows && seq_find(a.seqs, c1 - 1).start >= c0;
            __syncthreads();
        }
        float end[kAhead], sum[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (cb + i + 1 < a.nchunks) {  // the last chunk passes nothing on
                end[i] = a.hchunk[(cb + i) * total + e];
                sum[i] = a.schunk[(cb + i) * a.ch + d];
            }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t c = cb + i;
            if (c >= a.nchunks) break;
            if (at_e < total) a.hchunk[c * total + e] = in;
            if (c + 1 < a.nchunks) in = starts[c % 256] ? end[i] : fmaf(tc5::ex2(A * sum[i]), in, end[i]);
        }
    }
}

// ---- host ------------------------------------------------------------------------------------
int scan_check(const kda_scan_params &p);
// Arguments without chunk buffers and error word. `vec` covers u, dt, z and the given pointers.
ScanArgs scan_args(const kda_scan_params &p, const void *const *more, int n);

}  // namespace scan
}  // namespace kda
