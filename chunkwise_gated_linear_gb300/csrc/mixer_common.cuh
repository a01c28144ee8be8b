// Shared pieces of the token-mixer operators (kda_mixer.h): element and vector access,
// activations, packed-sequence lookup, packed fp32 pairs, scratch, and the sum of per-block
// partial results in a fixed order.
#pragma once

#include <cstdint>

#include "kda_common.cuh"
#include "kda_mixer.h"
#include "tc_util.cuh"

namespace kda {

// In kda_api.cu: the device error word of the current device, and the status of a CUDA result
// (kept for kda_status_string).
cudaError_t device_error_word(unsigned int **out);
int status_of_cuda(cudaError_t e);

namespace mix {

using bf16 = __nv_bfloat16;

// ---- element access -----------------------------------------------------------------------
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) {
    return x;
}
template <>
__device__ __forceinline__ bf16 from_f<bf16>(float x) {
    return __float2bfloat16_rn(x);
}

// ---- pairs of fp32 in one 64-bit register: two lanes of an FMA per instruction ---------------
using f2 = uint64_t;
__device__ __forceinline__ f2 pk(float lo, float hi) {
    f2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void upk(f2 v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }

// V consecutive elements as they lie in memory (V * sizeof(T) bytes, or one element).
template <typename T, int V>
struct Raw {
    static constexpr int kBytes = V * (int)sizeof(T);
    static constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
    uint32_t w[kWords];

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    // `p` aligned to min(16, kBytes). Plain loads: some inputs may be updated in place.
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i) {
                const uint4 q = reinterpret_cast<const uint4 *>(p)[i];
                w[4 * i] = q.x;
                w[4 * i + 1] = q.y;
                w[4 * i + 2] = q.z;
                w[4 * i + 3] = q.w;
            }
        } else if constexpr (kBytes == 8) {
            const uint2 q = *reinterpret_cast<const uint2 *>(p);
            w[0] = q.x;
            w[1] = q.y;
        } else if constexpr (kBytes == 4) {
            w[0] = *reinterpret_cast<const unsigned int *>(p);
        } else {
            static_assert(kBytes == 2, "one 16-bit element");
            w[0] = *reinterpret_cast<const unsigned short *>(p);
        }
    }
    // the first n of V elements, one by one, zeros after them; any element-aligned p
    __device__ __forceinline__ void load_some(const T *p, int n) {
        zero();
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (i < n) {
                if constexpr (sizeof(T) == 4)
                    w[i] = reinterpret_cast<const unsigned int *>(p)[i];
                else
                    w[i / 2] |= (uint32_t)reinterpret_cast<const unsigned short *>(p)[i] << (16 * (i & 1));
            }
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[i]);
        else
            return __uint_as_float((i & 1) ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
    }
    __device__ __forceinline__ f2 pair(int i) const { return pk(get(2 * i), get(2 * i + 1)); }
    __device__ __forceinline__ void unpack(float (&f)[V]) const {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = get(i);
    }
    __device__ __forceinline__ void pack(const float (&f)[V]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = __float_as_uint(f[i]);
        } else if constexpr (V == 1) {
            w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i)
                reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else if constexpr (kBytes == 8) {
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        } else if constexpr (kBytes == 4) {
            *reinterpret_cast<uint32_t *>(p) = w[0];
        } else {
            *reinterpret_cast<unsigned short *>(p) = (unsigned short)w[0];
        }
    }
    __device__ __forceinline__ void store_some(T *p, int n) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (i < n) {
                if constexpr (sizeof(T) == 4)
                    reinterpret_cast<uint32_t *>(p)[i] = w[i];
                else
                    reinterpret_cast<unsigned short *>(p)[i] = (unsigned short)(w[i / 2] >> (16 * (i & 1)));
            }
        }
    }
};

template <typename T, int V>
__device__ __forceinline__ void load_vec(float (&f)[V], const T *p) {
    Raw<T, V> r;
    r.load(p);
    r.unpack(f);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const float (&f)[V]) {
    Raw<T, V> r;
    r.pack(f);
    r.store(p);
}

// ---- activations --------------------------------------------------------------------------
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / (1 + e^-x): one exponential and one reciprocal on the special-function unit. Relative error below
// 4e-7, for negative x plus 8e-8 |x| (the exponent -x log2 e is rounded once); e^-x = inf gives 0.
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + tc5::ex2(-x * kLog2e)); }
// The value of the gate act(x), KDA_ACT_SILU or KDA_ACT_SIGMOID.
__device__ __forceinline__ float act_value(float x, bool silu) {
    const float s = sigmoid(x);
    return silu ? x * s : s;
}
// Its value and derivative.
__device__ __forceinline__ void act_both(float x, bool silu, float &val, float &der) {
    const float s = sigmoid(x);
    val = silu ? x * s : s;
    der = silu ? s * fmaf(x, 1.f - s, 1.f) : s * (1.f - s);
}

// ---- arithmetic on pairs -------------------------------------------------------------------
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ float hsum2(f2 v) {
    float lo, hi;
    upk(v, lo, hi);
    return lo + hi;
}
// 2^x of both halves
__device__ __forceinline__ f2 exp2_2(f2 v) {
    float lo, hi;
    upk(v, lo, hi);
    return pk(tc5::ex2(lo), tc5::ex2(hi));
}

// ---- sequences as row ranges ----------------------------------------------------------------
// Rows 0 .. rows - 1 hold the tokens of N sequences one after another: of T tokens each, or at
// the offsets cu[0 .. N] (cu != nullptr, rows == T).
struct Seqs {
    const int32_t *cu;
    int N, T;
    int64_t rows;
};
// The sequence of one row: start <= row < end whatever the offsets hold, s in [0, N).
struct SeqAt {
    int s;
    int64_t start, end;
};
__device__ __forceinline__ void seq_fill(const Seqs &q, int64_t row, SeqAt &at) {
    const int64_t b = q.cu[at.s], e = q.cu[at.s + 1];
    at.start = b < 0 ? 0 : (b > row ? row : b);
    at.end = e <= row ? row + 1 : (e > q.rows ? q.rows : e);
}
__device__ __forceinline__ SeqAt seq_find(const Seqs &q, int64_t row) {
    SeqAt at;
    if (q.cu == nullptr) {
        at.s = (int)(row / q.T);
        at.start = (int64_t)at.s * q.T;
        at.end = at.start + q.T;
        return at;
    }
    int lo = 0, hi = q.N - 1;  // the last s with cu[s] <= row
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (q.cu[mid] <= row)
            lo = mid;
        else
            hi = mid - 1;
    }
    at.s = lo;
    seq_fill(q, row, at);
    return at;
}
// The sequence that begins at row at.end (a row that exists); empty ones are stepped over.
__device__ __forceinline__ void seq_next(const Seqs &q, SeqAt &at) {
    const int64_t row = at.end;
    if (q.cu == nullptr) {
        ++at.s;
        at.start = row;
        at.end = row + q.T;
        return;
    }
    int s = at.s + 1 < q.N ? at.s + 1 : q.N - 1;
    while (s < q.N - 1 && q.cu[s + 1] <= row) ++s;
    at.s = s;
    seq_fill(q, row, at);
}
__device__ __forceinline__ bool seq_empty(const Seqs &q, int s) {
    return q.cu == nullptr ? q.T == 0 : q.cu[s] == q.cu[s + 1];
}
// One block checks the offsets and raises the error bit.
__device__ __forceinline__ void seq_check(const Seqs &q, unsigned int *err, int tid, int nthreads) {
    if (q.cu == nullptr) return;
    bool bad = false;
    for (int s = tid; s < q.N; s += nthreads) bad |= q.cu[s] > q.cu[s + 1];
    if (tid == 0) bad |= q.cu[0] != 0 || q.cu[q.N] != q.rows;
    if (bad) atomicOr(err, kDeviceErrSeqlens);
}

// ---- host side ------------------------------------------------------------------------------
inline bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The caller's workspace, or stream-ordered memory of the library's pool.
struct Scratch {
    void *ptr = nullptr;
    bool own = false;
    cudaStream_t stream = nullptr;
    cudaError_t get(void *given, size_t bytes, cudaStream_t s) {
        stream = s;
        if (bytes == 0) return cudaSuccess;
        if (given != nullptr) {
            ptr = given;
            return cudaSuccess;
        }
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        cudaMemPool_t pool = nullptr;
        if (e == cudaSuccess) e = scratch_pool(dev, &pool);
        if (e == cudaSuccess) e = cudaMallocFromPoolAsync(&ptr, bytes, pool, s);
        own = e == cudaSuccess;
        return e;
    }
    cudaError_t release(cudaError_t before) {
        if (!own) return before;
        own = false;
        const cudaError_t e = cudaFreeAsync(ptr, stream);
        return before != cudaSuccess ? before : e;
    }
};

// SMs of the current device (0 when it cannot be asked).
int sm_count();

// out[c] = sum over p of partial[p * total + c], in an order that the sizes alone fix (every 8th or 32nd part,
// then those sums); the columns go to up to four outputs one after another, an output that is null is left out.
struct SumOuts {
    float *out[4];
    int64_t len[4];
};
cudaError_t launch_sum_partials(const float *partial, int64_t parts, int64_t total, const SumOuts &outs, cudaStream_t stream);

}  // namespace mix
}  // namespace kda
