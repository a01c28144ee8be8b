// Attention over a paged cache, computed on the fp32 pipes: fp32 data (cache fp32 or 8-bit). See attn_common.cuh
// for how the work is cut.
//
// A unit is KEYS keys: lane (key, part) takes every (32 / KEYS)-th 16-byte chunk of its key against all query rows, the
// parts are added across lanes; then a lane owns DP / 32 neighbouring columns of O and goes through the keys. Arithmetic
// goes in pairs of fp32, without branches per row: rows that are not there are zeros (with a branch for each row the
// compiler keeps the rows' loads apart: 32768 tokens of 3 sequences, 4 key heads of 128, 135 us instead of 85, 70 % of what a
// copy moves). The rings fill the shared memory of an SM: two blocks of four warps, in fp32 above 128 channels one, over 8 bits with 4 rows up to
// 128 channels three.
#include <type_traits>

#include "attn_common.cuh"
#include "attn_launch.h"

namespace kda {
namespace attn {
namespace {

// N consecutive values of a row as pairs.
template <typename C, int N>
__device__ __forceinline__ void values(f2 (&x)[N / 2], const unsigned char *at) {
    if constexpr (sizeof(C) == 4) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 v = reinterpret_cast<const float2 *>(at)[i];
            x[i] = pk(v.x, v.y);
        }
    } else {
        Raw<uint16_t, N / 2> r;  // two values in each
        r.load(reinterpret_cast<const uint16_t *>(at));
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            float lo, hi;
            e4m3_to_f(r.w[i / 2] >> (16 * (i & 1)) & 0xffffu, lo, hi);
            x[i] = pk(lo, hi);
        }
    }
}

template <typename C, int DP, int RB, int KEYS, int SLOTS>
struct Fma {
    using S = Stream<C, DP, KEYS, SLOTS>;
    static constexpr int kParts = 32 / KEYS;
    static constexpr int kE = 16 / (int)sizeof(C);
    static constexpr int kCols = DP / 32;  // of a lane, side by side
    // shared memory: rings, q [warps][RB][DP], p [warps][KEYS][RB], rows' limits [warps][RB], the plan, exponent bytes
    static constexpr int kQ = kWarps * S::kBytes;
    static constexpr int kP = kQ + kWarps * RB * DP * 4;
    static constexpr int kLim = kP + kWarps * KEYS * RB * 4;
    static constexpr int kPlan = kLim + kWarps * RB * 4;
    static constexpr int kSc = kPlan + kPlanBytes;
    static constexpr int kSmem = kSc + kWarps * S::kScaleBytes;
    static_assert(kSmem <= 227 * 1024, "shared memory of a block");
    static constexpr int kFit = (228 * 1024) / (kSmem + 1024);
    static constexpr int kBlocks = kFit < 2 ? 1 : RB > 4 || kFit == 2 ? 2 : 3;
};

template <typename C, int DP, int RB, int KEYS, int SLOTS>
__global__ void __launch_bounds__(kThreads, Fma<C, DP, RB, KEYS, SLOTS>::kBlocks) attn_fma_kernel(const __grid_constant__ Args a) {
    using F = Fma<C, DP, RB, KEYS, SLOTS>;
    extern __shared__ __align__(128) unsigned char mem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    launch_dependents();
    Walk walk = find_walk<1>(a, reinterpret_cast<uint32_t *>(mem + F::kPlan));
    if (walk.left == 0) return;
    float *qs = reinterpret_cast<float *>(mem + F::kQ) + warp * RB * DP;
    float *pw = reinterpret_cast<float *>(mem + F::kP) + warp * KEYS * RB;
    int *lim = reinterpret_cast<int *>(mem + F::kLim) + warp * RB;
    unsigned char *own = mem + warp * F::S::kBytes;
    typename F::S st(a, own, mem + F::kSc + warp * F::S::kScaleBytes, lane, warp, walk);
    const int D = a.cache.D, key = lane & (KEYS - 1), part = lane / KEYS;
    const int cpr = D * (int)sizeof(C) / 16;

#pragma unroll 1
    while (walk.left > 0) {
        const Piece p = walk.piece(a);
        if (p.none()) {
            walk.step(a, p.weight);
            continue;
        }
#pragma unroll 1
        for (int r = 0; r < RB; ++r) {  // rows that are not there: zeros, which see nothing
            const float *from = static_cast<const float *>(a.q) + q_at(a, p, r < p.rows ? r : 0);
            for (int d = lane; d < DP; d += 32) qs[r * DP + d] = r < p.rows && d < D ? from[d] * a.scale_log2 : 0.f;
        }
        if (lane < RB) lim[lane] = lane < p.rows ? seen(a, p.len, p.row0 + lane) : 0;
        __syncwarp();
        const int least = lim[0];  // keys from here on are not seen by all its rows
        float m[RB], l[RB];
        f2 acc[RB][F::kCols / 2];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int j = 0; j < F::kCols / 2; ++j) acc[r][j] = pk(0.f, 0.f);
        }
#pragma unroll 1
        for (uint32_t u = p.u0; u < p.u1; ++u) {
            const int pos0 = (int)u * KEYS;
            st.template ready<false>();
            if (pos0 < p.last) {  // the same for the whole warp
                const unsigned char *ks = own + st.slot * F::S::kSlot;
                const uint8_t *sc = st.bytes();
                f2 dots[RB];
#pragma unroll
                for (int r = 0; r < RB; ++r) dots[r] = pk(0.f, 0.f);
#pragma unroll 4
                for (int c = part; c < cpr; c += F::kParts) {
                    f2 kf[F::kE / 2];
                    values<C, F::kE>(kf, ks + key * F::S::kPitch + ((c ^ (key & 7)) << 4));
#pragma unroll
                    for (int r = 0; r < RB; ++r) {
#pragma unroll
                        for (int e = 0; e < F::kE; e += 4) {
                            const float4 qv = *reinterpret_cast<const float4 *>(qs + r * DP + c * F::kE + e);
                            dots[r] = fma2(kf[e / 2], pk(qv.x, qv.y), dots[r]);
                            dots[r] = fma2(kf[e / 2 + 1], pk(qv.z, qv.w), dots[r]);
                        }
                    }
                }
                float x[RB];
#pragma unroll
                for (int r = 0; r < RB; ++r) x[r] = hsum2(dots[r]);
                float kscale = 1.f, vscale = 1.f;
                if constexpr (F::S::kScaled) {
                    kscale = __uint_as_float((uint32_t)sc[key] << 23);
                    vscale = __uint_as_float((uint32_t)sc[KEYS + key] << 23);
                }
                const int pos = pos0 + key;
                bool grew = false;
                float alpha[RB];
#pragma unroll
                for (int r = 0; r < RB; ++r) {
                    alpha[r] = 1.f;
#pragma unroll
                    for (int o = KEYS; o < 32; o <<= 1) x[r] += __shfl_xor_sync(0xffffffffu, x[r], o);
                    x[r] = pos < lim[r] ? x[r] * kscale : -INFINITY;
                    float top = x[r];
#pragma unroll
                    for (int o = 1; o < KEYS; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    if (top > m[r]) {
                        alpha[r] = tc5::ex2(m[r] - top);
                        m[r] = top;
                        grew = true;
                    }
                    // no key seen so far: 2^(-inf - 0) = 0
                    const float w = tc5::ex2(x[r] - (m[r] == -INFINITY ? 0.f : m[r]));
                    l[r] = l[r] * alpha[r] + (part == 0 ? w : 0.f);
                    if (part == 0) pw[key * RB + r] = w * vscale;
                }
                __syncwarp();
                if (grew) {
#pragma unroll
                    for (int r = 0; r < RB; ++r)
#pragma unroll
                        for (int j = 0; j < F::kCols / 2; ++j) acc[r][j] = mul2(acc[r][j], pk(alpha[r], alpha[r]));
                }
            }
            st.template release<false>();
            st.template ready<true>();
            if (pos0 < p.last) {
                const unsigned char *vs = own + st.slot * F::S::kSlot;
                auto add = [&](int k, auto all) {
                    f2 v[F::kCols / 2];
                    constexpr int kBytes = F::kCols * (int)sizeof(C), kStep = kBytes < 16 ? kBytes : 16, kN = kStep / (int)sizeof(C);
#pragma unroll
                    for (int h = 0; h < kBytes / kStep; ++h) {
                        const int byte = lane * kBytes + h * kStep;
                        f2 t[kN / 2];
                        values<C, kN>(t, vs + k * F::S::kPitch + ((((byte >> 4) ^ (k & 7)) << 4) | (byte & 15)));
#pragma unroll
                        for (int i = 0; i < kN / 2; ++i) v[h * kN / 2 + i] = t[i];
                    }
                    float w[RB];
                    load_vec<float, RB>(w, pw + k * RB);
#pragma unroll
                    for (int r = 0; r < RB; ++r) {
                        // a value that this row does not see must not reach it, not even times zero
                        if (!decltype(all)::value && pos0 + k >= lim[r]) continue;
#pragma unroll
                        for (int j = 0; j < F::kCols / 2; ++j) acc[r][j] = fma2(pk(w[r], w[r]), v[j], acc[r][j]);
                    }
                };
                if (pos0 + KEYS <= least) {
#pragma unroll 4
                    for (int k = 0; k < KEYS; ++k) add(k, std::true_type{});
                } else {
#pragma unroll 1
                    for (int k = 0; k < KEYS; ++k) add(k, std::false_type{});
                }
            }
            st.template release<true>();
        }
        float *piece = piece_mem(a, blockIdx.x * kWarps + warp, p.u0 == 0);
        if (lane == 0) tell_ends(a, p, blockIdx.x * kWarps + warp);
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            if (r >= p.rows) break;
            float t = l[r];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            const bool whole = p.whole();
            const int64_t row = out_row(a, p, r);
            const bool empty = whole && t == 0.f;  // zeros, whatever the values are
            const float f = whole ? 1.f / t : 1.f;
            float *to = whole ? static_cast<float *>(a.o) + row * D : piece + r * D;
#pragma unroll
            for (int j = 0; j < F::kCols / 2; ++j) {
                const int d = lane * F::kCols + 2 * j;
                float lo, hi;
                upk(mul2(acc[r][j], pk(f, f)), lo, hi);
                if (d < D) *reinterpret_cast<float2 *>(to + d) = empty ? make_float2(0.f, 0.f) : make_float2(lo, hi);
            }
            if (lane == 0) {
                if (!whole)
                    reinterpret_cast<float2 *>(piece + a.rows * D)[r] = make_float2(m[r], t);
                else if (a.lse != nullptr)
                    a.lse[row] = lse_of(m[r], t);
            }
        }
        __syncwarp();
        walk.step(a, p.weight);
    }
    copies_wait<0>();
}

template <typename C, int DP, int RB, int KEYS, int SLOTS>
struct Variant {
    using F = Fma<C, DP, RB, KEYS, SLOTS>;
    static cudaError_t launch(const Args &a, cudaStream_t stream) {
        return launch_kernel<attn_fma_kernel<C, DP, RB, KEYS, SLOTS>, F::kSmem, 1>(a, stream);
    }
    static int workers() { return F::kBlocks * kWarps; }
    static int unit() { return KEYS; }
};
// Calls f with the variant for these sizes. Keys of a unit: 16, or 8 where an fp32 ring of such units would leave one block. Slots of a ring: in
// fp32 as many as leave room for two blocks on an SM up to 128 channels, and five in one block above; over 8 bits, which leave room
// for two blocks or more, five or six, and four above 128 channels. (us, with one slot less and one more; 3 sequences of 32768, 16384 or 8192
// tokens for 64, 128 and 256 channels, 4 key heads, 4 rows and 8 rows: fp32 50 (50, 71), 74 (74, 105); 52 (54, 57), 84 (83, 107);
// 54 (53, 55), 79 (78, 82); 8 bits 43 (43, 43), 71 (71, 71); 38 (38, 38), 62 (62, 63); 34 and, with five, 35; 55 and, with five, 60.)
template <typename C, int RB, typename F>
auto pick(const Args &a, F f) {
    constexpr bool k4 = sizeof(C) == 4;
    if (a.cache.D <= 64) return f(Variant<C, 64, RB, 16, 6>{});
    if (a.cache.D <= 128) return f(Variant<C, 128, RB, (k4 && RB > 4) ? 8 : 16, (k4 && RB == 4) ? 3 : 5>{});
    return f(Variant<C, 256, RB, k4 ? 8 : 16, k4 ? 5 : 4>{});
}
template <typename F>
auto pick(const Args &a, F f) {
    if (a.cache.ks != nullptr) return a.rows == 4 ? pick<uint8_t, 4>(a, f) : pick<uint8_t, 8>(a, f);
    return a.rows == 4 ? pick<float, 4>(a, f) : pick<float, 8>(a, f);
}

}  // namespace

// Query rows read from shared memory for every key are what bounds more than four of them (32768 tokens of 3 sequences, 4 key heads of
// 128: 85 us for 4 rows, in items of 16 274; 129 for 8; for 16 rows 220 as two items of 8, 258 as four of 4, 318 as one).
int fma_rows(int all) { return all <= 4 ? 4 : 8; }
int fma_unit_shift(const Args &a) {
    return pick(a, [](auto v) { return decltype(v)::unit() == 16 ? 4 : 3; });
}
int fma_workers(const Args &a) {
    return pick(a, [](auto v) { return decltype(v)::workers(); });
}
cudaError_t launch_attn_fma(const Args &a, cudaStream_t stream) {
    return pick(a, [&](auto v) { return decltype(v)::launch(a, stream); });
}

}  // namespace attn
}  // namespace kda
