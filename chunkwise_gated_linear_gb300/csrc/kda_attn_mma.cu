// Attention over a paged cache, computed by matrix instructions: bf16 queries, cache bf16 or 8-bit. See attn_common.cuh for
// how the work is cut and how keys and values stream in.
//
// Few query rows meet many keys, so the keys are the long side M of the instructions (m16n8k16) and 8 NT query rows the
// short side N: S^T = K Q^T (16 keys x rows), O^T += V^T P^T (channels x rows). K is read from the ring as it lies, V
// through the transposing load; the accumulator of S^T becomes the operand P^T by a transpose of 8 x 8 blocks
// in registers. A row's statistics are shared by the 8 lanes that hold its keys, but the sum is kept per
// lane and the reference m of the exponentials moves only when a score of the row is more than 8 (base 2) above it, so that
// most steps exchange nothing between lanes.
//
// Probabilities are rounded to bf16, the one type that a product with bf16 values takes; the sum l is not. Against 64 bits the
// result for 131071 tokens is off by 2.4e-3 of its norm, with fp32 probabilities by 1.7e-3, which is the rounding of the result.
// A second product with what that rounding left would take it back at as many matrix instructions again.
//
// What bounds it is the stream of keys and values where they are many: 64 sequences of up to 16384 tokens, 8 key heads of 128 in
// 8 bits, 187 us, 95 % of what a copy moves (three blocks of four warps on an SM, each warp 24 KB ahead; tensor pipes 18 % busy,
// so larger matrix instructions would change nothing); one sequence of 131071 in bf16 92 us, 86 % with the start and
// the join. With many rows it is the instructions, 680 for a warp's 32 keys and 8 rows in 8 bits (all of a launch's over the
// number of such units): 4 new tokens of 8 heads a key head, 16 sequences of up to 8192: 41 us, 24 %. 64 rows of 128 channels
// have more live than the registers of three blocks hold (172 bytes spilled over 8 bits, 72 in bf16; elsewhere at most 68).
//
// 8-bit cache: e4m3 numbers are exact in fp16, so K and V are widened in registers and the products run in fp16
// (one conversion per two numbers; widening to bf16 takes four to five instructions). Q goes to fp16 times a power of two per
// row that puts its largest entry at 2^14: entries down to 2^-28 of it stay exact. The power of two of a key multiplies
// its scores, that of a value its probability: P' = 2^(score + sv - M) with a reference M of its own, between 2^-24 and
// 2^14 in fp16 (11 bits), while the sum l keeps the plain 2^(score - m). M is kept as M - m: beside a large score a value's
// power of two would be lost. Both references are watched by one
// comparison per score, with min(m + 8, M + 14 - the largest sv so far). That sv may belong to a key of no weight, and then
// each unit takes the longer way without a move (a value 2^6 to 2^14 above the others and of no weight in every 64 keys: 64
// sequences of up to 16384 tokens 178 us instead of 173, the new tokens above 45 to 46 instead of 41).
#include <type_traits>

#include "attn_common.cuh"
#include "attn_launch.h"

namespace kda {
namespace attn {
namespace {

constexpr float kGrow = 8.f;  // a score may pass its reference by so much before it moves: exponentials up to 2^8
constexpr float kMost = 14.f;  // 8-bit: P' up to 2^14, within fp16
constexpr float kWatch = kMost - 0.01f;  // looked after from here on, so that no rounding hides what passes kMost

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(x));
    return d;
}
// Bytes 0, 1 and bytes 2, 3 of x as two halves each.
__device__ __forceinline__ void widen(uint32_t x, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

template <typename C, int DP, int NT, int SLOTS, int TEAM>
struct Mma {
    static constexpr bool kScaled = sizeof(C) == 1;
    static constexpr int kJoint = kScaled || TEAM > 1 ? 2 : 1;  // blocks of 16 keys in a unit
    static constexpr int kKeys = 16 * kJoint;
    using S = Stream<C, DP, kKeys, SLOTS, TEAM>;
    static constexpr int kSteps = DP / 16;  // products of S^T, and blocks of 16 channels of O^T
    static constexpr int kRows = 8 * NT;  // of a warp
    static constexpr int kQBytes = NT * kSteps * 256;  // Q^T of a warp: [NT][kSteps][32 lanes] of 8 bytes
    static constexpr int kStats = 4 * kRows;           // floats of a warp: what a score is multiplied with, m, M, a factor
    // shared memory: rings, Q^T, statistics, the plan, exponent bytes
    static constexpr int kWorkers = kWarps / TEAM;
    static constexpr int kQ = kWorkers * S::kBytes;
    static constexpr int kStat = kQ + kWarps * kQBytes;
    static constexpr int kPlan = kStat + kWarps * kStats * 4;
    static constexpr int kSc = kPlan + kPlanBytes;
    static constexpr int kSmem = kSc + kWorkers * S::kScaleBytes;
    static constexpr int kFit = (228 * 1024) / (kSmem + 1024);
    // registers: O^T is 4 kSteps NT of a lane's, the scores 4 kJoint NT
    static constexpr int kLive = 4 * kSteps * NT + 4 * kJoint * NT + 8 * NT + 72;
    static constexpr int kByRegs = 65536 / (kThreads * (kLive < 96 ? 96 : kLive > 255 ? 255 : kLive));
    static constexpr int kBlocks = kFit < kByRegs ? kFit : kByRegs;
};

// The largest of each of 2 NT values over the 8 lanes g: of value i it ends in the lanes with i in the upper bits of g (lane
// bits 4, 3, 2). Half of the values go to the other lane in each step, while there are two or more.
template <int N>
__device__ __forceinline__ float spread_max(float (&v)[N], int lane) {
    int n = N;
#pragma unroll
    for (int bit = 16; bit >= 4; bit >>= 1) {
        const bool up = lane & bit;
        if (n > 1) {
            n /= 2;
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (i < n) {
                    const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                    v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, bit));
                }
        } else {
            v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], bit));
        }
    }
    return v[0];
}

// What is done once per piece is kept short (loops, statistics in shared memory while they change): code that runs once
// is bound by fetching it, about 40 cycles for an instruction (16 sequences with four drafted tokens each: 119 us
// with everything unrolled).
template <typename C, int DP, int NT, int SLOTS, int TEAM>
__global__ void __launch_bounds__(kThreads, Mma<C, DP, NT, SLOTS, TEAM>::kBlocks) attn_mma_kernel(const __grid_constant__ Args a) {
    using M = Mma<C, DP, NT, SLOTS, TEAM>;
    using S = typename M::S;
    constexpr int kSteps = M::kSteps, kJoint = M::kJoint, kKeys = M::kKeys, kRows = M::kRows;
    extern __shared__ __align__(1024) unsigned char mem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    launch_dependents();
    Walk walk = find_walk<TEAM>(a, reinterpret_cast<uint32_t *>(mem + M::kPlan));
    if (walk.left == 0) return;  // the whole team
    const int worker = warp / TEAM;
    unsigned char *own = mem + worker * S::kBytes;
    S st(a, own, mem + M::kSc + worker * S::kScaleBytes, lane, warp, walk);
    uint2 *qmem = reinterpret_cast<uint2 *>(mem + M::kQ + warp * M::kQBytes) + lane;  // [NT][kSteps], 32 apart
    // of each row: what its scores are multiplied with, the reference m, M - m, the factor of the last move
    float *stats = reinterpret_cast<float *>(mem + M::kStat) + warp * M::kStats;
    float *row_m = stats + kRows, *row_mv = row_m + kRows, *row_back = row_mv + kRows;
    const int D = a.cache.D;
    // the row whose statistics this lane moves: of value i = 2 n + j, in the order of spread_max
    const int my_i = g >> (NT == 4 ? 0 : NT == 2 ? 1 : 2), my_row = 8 * (my_i >> 1) + 2 * c + (my_i & 1);

#pragma unroll 1
    while (walk.left > 0) {
        Piece p = walk.piece(a);
        if (p.none()) {
            walk.step(a, p.weight);
            continue;
        }
        if constexpr (TEAM > 1) p.mine(a, warp % TEAM * kRows, kRows);
        // Q^T: row 8 n + g, the lane's channels of each block of 16 in the order in which K's come out of the ring
#pragma unroll 1
        for (int n = 0; n < NT; ++n) {
            const bool there = 8 * n + g < p.rows;
            const bf16 *from = static_cast<const bf16 *>(a.q) + (there ? q_at(a, p, 8 * n + g) : 0) + (M::kScaled ? 4 * c : 2 * c);
            uint2 x[kSteps];
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                x[k] = make_uint2(0u, 0u);
                if (there && 16 * k < D) {
                    if constexpr (M::kScaled)
                        x[k] = *reinterpret_cast<const uint2 *>(from + 16 * k);
                    else
                        x[k] = make_uint2(*reinterpret_cast<const uint32_t *>(from + 16 * k), *reinterpret_cast<const uint32_t *>(from + 16 * k + 8));
                }
            }
            float by = a.scale_log2;
            if constexpr (M::kScaled) {
                float top = 0.f;
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    top = fmaxf(top, fmaxf(finite_abs(__uint_as_float(x[k].x << 16)), finite_abs(__uint_as_float(x[k].x & 0xffff0000u))));
                    top = fmaxf(top, fmaxf(finite_abs(__uint_as_float(x[k].y << 16)), finite_abs(__uint_as_float(x[k].y & 0xffff0000u))));
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // 2^e with the largest entry at 2^14 .. 2^15, within what fp32 holds
                int e = 127 + 14 - (int)(__float_as_uint(top) >> 23);
                e = e > 126 ? 126 : e;
                const float up = pow2(e);
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    x[k].x = pack_f16(__uint_as_float(x[k].x << 16) * up, __uint_as_float(x[k].x & 0xffff0000u) * up);
                    x[k].y = pack_f16(__uint_as_float(x[k].y << 16) * up, __uint_as_float(x[k].y & 0xffff0000u) * up);
                }
                by *= pow2(-e);
            }
#pragma unroll
            for (int k = 0; k < kSteps; ++k) qmem[(n * kSteps + k) * 32] = x[k];
            if (c == 0) stats[8 * n + g] = by;
        }
        const int least = seen(a, p.len, p.row0);  // keys from here on are not seen by all rows
        __syncwarp();

        float o[kSteps][NT][4];
        // of rows 8 n + 2 c, + 1: factor of the scores, -m, the sum of the exponentials, 8-bit: 2^(m - M); the score at which m
        // or M moves (-infinity: nothing seen yet)
        f2 rowf[NT], ref[NT], l[NT], turn[NT];
        float lim[NT][2];
        float sv_top = -127.f;      // 8-bit: the largest exponent of a value so far
        bool nothing = true;        // of this lane's row my_row: nothing seen yet
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float2 by = *reinterpret_cast<const float2 *>(stats + 8 * n + 2 * c);
            rowf[n] = pk(by.x, by.y);
            ref[n] = l[n] = pk(0.f, 0.f);
            turn[n] = pk(1.f, 1.f);
            lim[n][0] = lim[n][1] = -INFINITY;
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[k][n][i] = 0.f;
        }
        float my_m = 0.f, my_mv = 0.f;  // of my_row: m, and 8-bit M - m
        // -m of all rows, after it has moved
        auto references = [&] {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 m2 = *reinterpret_cast<const float2 *>(row_m + 8 * n + 2 * c);
                ref[n] = pk(m2.x == -INFINITY ? 0.f : -m2.x, m2.y == -INFINITY ? 0.f : -m2.y);
            }
        };
        // the borders of all rows, after the references or sv_top have moved; rounded down, so that a score that has to move a
        // reference is seen whatever its size
        auto borders = [&](bool moved) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 m2 = *reinterpret_cast<const float2 *>(row_m + 8 * n + 2 * c);
                float over[2] = {kGrow, kGrow};
                if constexpr (M::kScaled) {
                    const float2 v2 = *reinterpret_cast<const float2 *>(row_mv + 8 * n + 2 * c);
                    over[0] = fminf(kGrow, v2.x + kWatch - sv_top);
                    over[1] = fminf(kGrow, v2.y + kWatch - sv_top);
                    if (moved) turn[n] = pk(tc5::ex2(-v2.x), tc5::ex2(-v2.y));
                }
                lim[n][0] = __fadd_rd(m2.x, over[0]);
                lim[n][1] = __fadd_rd(m2.y, over[1]);
            }
        };
        if (lane < kRows) {
            row_m[lane] = -INFINITY;
            row_mv[lane] = 0.f;
        }

#pragma unroll 1
        for (uint32_t u = p.u0; u < p.u1; ++u) {
            st.template ready<false>();
            const int pos0 = (int)u * kKeys;
            const bool count = pos0 < p.last;  // the same for the whole warp
            float x[kJoint][NT][4];
            if (count) {
                const uint32_t krow = st.oldest() + (lane & 15) * S::kPitch;
#pragma unroll
                for (int h = 0; h < kJoint; ++h)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[h][n][i] = 0.f;
                // few rows: sums of even and odd steps, so that half as many products wait for one another
                constexpr bool kTwo = NT * kJoint == 1;
                float x2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < kSteps; k += M::kScaled ? 2 : 1) {
                    uint32_t f[kJoint][M::kScaled ? 2 : 1][4];
#pragma unroll
                    for (int h = 0; h < kJoint; ++h) {
                        if constexpr (M::kScaled) {
                            // 16-byte chunks k and k + 1 are channels 16 k .. 16 k + 31: keys g and g + 8, channels 4 c .. 4 c + 3 of each
                            uint32_t r[4];
                            ldsm(r, krow + 16 * h * S::kPitch + (((k + (lane >> 4)) ^ (lane & 7)) << 4));
                            widen(r[0], f[h][0][0], f[h][0][2]);
                            widen(r[1], f[h][0][1], f[h][0][3]);
                            widen(r[2], f[h][1][0], f[h][1][2]);
                            widen(r[3], f[h][1][1], f[h][1][3]);
                        } else {
                            ldsm(f[h][0], krow + 16 * h * S::kPitch + (((2 * k + (lane >> 4)) ^ (lane & 7)) << 4));
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int t = 0; t < (M::kScaled ? 2 : 1); ++t) {
                            const uint2 qv = qmem[(n * kSteps + k + t) * 32];
#pragma unroll
                            for (int h = 0; h < kJoint; ++h) {
                                if constexpr (M::kScaled)
                                    mma_f16(x[h][n], f[h][t], qv.x, qv.y);
                                else
                                    mma_bf16(kTwo && (k & 1) ? x2 : x[h][n], f[h][t], qv.x, qv.y);
                            }
                        }
                }
                if constexpr (kTwo) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[0][0][i] += x2[i];
                }
            }
            st.template release<false>();
            uint32_t pb[kJoint][NT][2];
            bool edge = false;
            if (count) {
                // scores, base 2; element i of block h: key 16 h + g + 8 (i / 2), row 8 n + 2 c + i % 2
                float fv[kJoint][2];  // 8-bit: the values' powers of two
                edge = pos0 + kKeys > least;
                if constexpr (M::kScaled) {
                    const uint8_t *sc = st.bytes();
                    // an exponent above all others moves the borders; keys that no row sees have old bytes or none, which only lower them
                    const float top = (float)((int)__reduce_max_sync(0xffffffffu, (uint32_t)sc[kKeys + lane]) - 127);
                    if (top > sv_top) {
                        sv_top = top;
                        borders(false);
                    }
#pragma unroll
                    for (int h = 0; h < kJoint; ++h)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float fk = __uint_as_float((uint32_t)sc[16 * h + g + 8 * i] << 23);
                            fv[h][i] = __uint_as_float((uint32_t)sc[kKeys + 16 * h + g + 8 * i] << 23);
#pragma unroll
                            for (int n = 0; n < NT; ++n)  // the row's factor first: times a large power of two it could pass fp32 where the sum is 0
                                upk(mul2(mul2(pk(x[h][n][2 * i], x[h][n][2 * i + 1]), rowf[n]), pk(fk, fk)), x[h][n][2 * i], x[h][n][2 * i + 1]);
                        }
                } else {
#pragma unroll
                    for (int h = 0; h < kJoint; ++h)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i) upk(mul2(pk(x[h][n][2 * i], x[h][n][2 * i + 1]), rowf[n]), x[h][n][2 * i], x[h][n][2 * i + 1]);
                }
                if (edge) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int end = seen(a, p.len, p.row0 + 8 * n + 2 * c + j) - pos0 - g;
#pragma unroll
                            for (int h = 0; h < kJoint; ++h) {
                                if (end <= 16 * h) x[h][n][j] = -INFINITY;
                                if (end <= 16 * h + 8) x[h][n][j + 2] = -INFINITY;
                            }
                        }
                }
                bool grows = false;
#pragma unroll
                for (int h = 0; h < kJoint; ++h)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) grows |= x[h][n][i] > lim[n][i & 1];
                if (__any_sync(0xffffffffu, grows)) {
                    // A reference moves up, never down, and by what its own row sees alone, so that a row's result does not follow, not
                    // even in its roundings, from the others of the warp. With nothing seen yet l and O are 0.
                    float v[2 * NT];
#pragma unroll
                    for (int i = 0; i < 2 * NT; ++i) {
                        v[i] = fmaxf(x[0][i / 2][i & 1], x[0][i / 2][(i & 1) + 2]);
                        if constexpr (kJoint == 2) v[i] = fmaxf(v[i], fmaxf(x[1][i / 2][i & 1], x[1][i / 2][(i & 1) + 2]));
                    }
                    const float top = spread_max(v, lane);
                    float back = 1.f;
                    const bool first = nothing;
                    if (first ? top > -INFINITY : top - my_m > kGrow) {
                        back = first ? 0.f : tc5::ex2(my_m - top);
                        my_mv -= first ? 0.f : top - my_m;
                        my_m = top;
                        nothing = false;
                    }
                    row_m[my_row] = nothing ? -INFINITY : my_m;
                    (M::kScaled ? stats : row_back)[my_row] = back;
                    __syncwarp();
                    references();
                    if constexpr (M::kScaled) {
                        // from the differences to m, as the scores may be so large that a value's power of two is lost beside them
                        float ev[kJoint][2];
#pragma unroll
                        for (int h = 0; h < kJoint; ++h)
#pragma unroll
                            for (int i = 0; i < 2; ++i) ev[h][i] = (float)((int)(__float_as_uint(fv[h][i]) >> 23) - 127);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float y[2] = {-INFINITY, -INFINITY};
#pragma unroll
                            for (int h = 0; h < kJoint; ++h)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    float lo, hi;
                                    upk(add2(pk(x[h][n][2 * i], x[h][n][2 * i + 1]), ref[n]), lo, hi);
                                    y[0] = fmaxf(y[0], lo + ev[h][i]);
                                    y[1] = fmaxf(y[1], hi + ev[h][i]);
                                }
                            v[2 * n] = y[0];
                            v[2 * n + 1] = y[1];
                        }
                        // the largest P' at 2^6, so that none passes 2^kMost soon; rows of zeros (sv = -126) alone leave it lower, or
                        // 2^(score - M), with a score of up to m + 8, would pass what fp32 holds
                        const float top_v = spread_max(v, lane);
                        back = 1.f;
                        if (!nothing) {
                            const float to = fmaxf(first || top_v > my_mv + kMost ? top_v - 6.f : my_mv, -119.f);
                            back = first ? 0.f : tc5::ex2(my_mv - to);
                            my_mv = to;
                        }
                        row_mv[my_row] = my_mv;
                        row_back[my_row] = back;
                        __syncwarp();
                    }
                    borders(true);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float2 b2 = *reinterpret_cast<const float2 *>(row_back + 8 * n + 2 * c);
                        const f2 f = pk(b2.x, b2.y);
                        if constexpr (M::kScaled) {
                            const float2 l2 = *reinterpret_cast<const float2 *>(stats + 8 * n + 2 * c);
                            l[n] = mul2(l[n], pk(l2.x, l2.y));
                        } else {
                            l[n] = mul2(l[n], f);
                        }
#pragma unroll
                        for (int k = 0; k < kSteps; ++k)
#pragma unroll
                            for (int i = 0; i < 2; ++i) upk(mul2(pk(o[k][n][2 * i], o[k][n][2 * i + 1]), f), o[k][n][2 * i], o[k][n][2 * i + 1]);
                    }
                    __syncwarp();
                }
#pragma unroll
                for (int h = 0; h < kJoint; ++h)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            f2 w = exp2_2(add2(pk(x[h][n][2 * i], x[h][n][2 * i + 1]), ref[n]));
                            l[n] = add2(l[n], w);
                            // in this order: w turn is P' without the value's power of two, at most 2^127 and 0 for a key that is not seen; turn fv
                            // alone passes what fp32 holds where the powers of two lie far apart (2^120 beside an infinity)
                            if constexpr (M::kScaled) w = mul2(mul2(w, turn[n]), pk(fv[h][i], fv[h][i]));
                            float lo, hi;
                            upk(w, lo, hi);
                            pb[h][n][i] = transpose8(M::kScaled ? pack_f16(lo, hi) : pack_bf16(lo, hi));
                        }
            }
            st.template ready<true>();
            if (count) {
                const uint32_t vs = st.oldest();
                // O^T += V^T P^T, for all rows, or those of one token alone, from the values at its first `end` keys
                auto values = [&](auto all, int token, int end) {
#pragma unroll
                    for (int h = 0; h < kJoint; ++h) {
                        const uint32_t vrow = vs + (16 * h + (M::kScaled ? lane & 15 : (lane & 7) + ((lane >> 4) << 3))) * S::kPitch;
#pragma unroll
                        for (int k = 0; k < kSteps; k += M::kScaled ? 2 : 1) {
                            uint32_t r[4], f[2][4];
                            if constexpr (M::kScaled) {
                                // 16 keys x 16-byte chunks k, k + 1, transposed in units of two bytes: channels 2 g, 2 g + 1 of keys 2 c, 2 c + 1;
                                // bytes (key 2c, channel 2g), (2c, 2g + 1), (2c + 1, 2g), (2c + 1, 2g + 1): pair the keys
                                ldsm_t(r, vrow + (((k + (lane >> 4)) ^ (lane & 7)) << 4));
#pragma unroll
                                for (int t = 0; t < 2; ++t) {
                                    widen(__byte_perm(r[2 * t], 0, 0x3120), f[t][0], f[t][1]);
                                    widen(__byte_perm(r[2 * t + 1], 0, 0x3120), f[t][2], f[t][3]);
                                }
                            } else {
                                ldsm_t(f[0], vrow + (((2 * k + ((lane >> 3) & 1)) ^ (lane & 7)) << 4));
                            }
                            if constexpr (!decltype(all)::value) {
                                // registers 0, 1: keys 2 c, 2 c + 1; 2, 3: eight further on
                                const int e = end - 16 * h - 2 * c;
                                const uint32_t near = e <= 0 ? 0u : e == 1 ? 0xffffu : ~0u, far = e <= 8 ? 0u : e == 9 ? 0xffffu : ~0u;
#pragma unroll
                                for (int t = 0; t < (M::kScaled ? 2 : 1); ++t)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) f[t][i] &= i < 2 ? near : far;
                            }
#pragma unroll
                            for (int t = 0; t < (M::kScaled ? 2 : 1); ++t)
#pragma unroll
                                for (int n = 0; n < NT; ++n) {
                                    if constexpr (decltype(all)::value) {
                                        if constexpr (M::kScaled)
                                            mma_f16(o[k + t][n], f[t], pb[h][n][0], pb[h][n][1]);
                                        else
                                            mma_bf16(o[k + t][n], f[t], pb[h][n][0], pb[h][n][1]);
                                    } else {
                                        // added up as above, so that such a value changes no rounding either
                                        float sum[4] = {o[k + t][n][0], o[k + t][n][1], o[k + t][n][2], o[k + t][n][3]};
                                        if constexpr (M::kScaled)
                                            mma_f16(sum, f[t], pb[h][n][0], pb[h][n][1]);
                                        else
                                            mma_bf16(sum, f[t], pb[h][n][0], pb[h][n][1]);
#pragma unroll
                                        for (int i = 0; i < 4; ++i)
                                            if ((unsigned)(p.row0 + 8 * n + 2 * c + (i & 1) - token * a.group) < (unsigned)a.group) o[k + t][n][i] = sum[i];
                                    }
                                }
                        }
                    }
                };
                bool odd = false;
                if (edge && a.T > 1) {  // is any value not finite?
#pragma unroll 1
                    for (uint32_t w = 16 * lane; w < (uint32_t)S::kSlot; w += 512) {
                        const uint4 q4 = *reinterpret_cast<const uint4 *>(own + (vs - st.ring) + w);
                        const uint32_t q[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            // all bits of an exponent (8-bit: of a number without its sign) set: adding the lowest of them carries out
                            if constexpr (M::kScaled)
                                odd |= (((q[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
                            else
                                odd |= (((q[i] & 0x7f807f80u) + 0x00800080u) & 0x80008000u) != 0;
                        }
                    }
                    odd = __any_sync(0xffffffffu, odd);
                }
                if (!odd) {
                    values(std::true_type{}, 0, 0);
                } else {
                    // Such a value would reach rows that do not see its key, as 0 * NaN: one token's rows at a time, the values that it
                    // does not see taken as zeros.
#pragma unroll 1
                    for (int t = token_of(a, p.row0); t <= token_of(a, p.row0 + p.rows - 1); ++t) values(std::false_type{}, t, p.len - a.T + t + 1 - pos0);
                }
            }
            st.template release<true>();
        }

        // of the worker's rows, this warp's begin at `base`
        const int base = TEAM > 1 ? warp % TEAM * kRows : 0;
        float *piece = piece_mem(a, blockIdx.x * M::kWorkers + worker, p.u0 == 0);
        const bool whole = p.whole();
        if (warp % TEAM == 0 && lane == 0) tell_ends(a, p, blockIdx.x * M::kWorkers + worker);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float sum[2];
            upk(l[n], sum[0], sum[1]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], d);
                const int r = 8 * n + 2 * c + j;
                if (r >= p.rows) continue;
                const float top = row_m[r];
                float f = M::kScaled ? tc5::ex2(row_mv[r]) : 1.f;
                const bool empty = whole && sum[j] == 0.f;  // zeros, whatever the values are
                if (whole) f = f / sum[j];
                const int64_t row = out_row(a, p, r);
                bf16 *to = static_cast<bf16 *>(a.o) + row * D;
                float *part = piece + (base + r) * D;
                if (g == 0) {
                    if (!whole)
                        reinterpret_cast<float2 *>(piece + a.rows * D)[base + r] = make_float2(top, sum[j]);
                    else if (a.lse != nullptr)
                        a.lse[row] = lse_of(top, sum[j]);
                }
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    if (16 * k >= D) break;
                    const float lo = empty ? 0.f : o[k][n][j] * f, hi = empty ? 0.f : o[k][n][j + 2] * f;
                    if constexpr (M::kScaled) {
                        if (whole)
                            *reinterpret_cast<uint32_t *>(to + 16 * k + 2 * g) = pack_bf16(lo, hi);
                        else
                            *reinterpret_cast<float2 *>(part + 16 * k + 2 * g) = make_float2(lo, hi);
                    } else if (whole) {
                        to[16 * k + g] = from_f<bf16>(lo);
                        to[16 * k + g + 8] = from_f<bf16>(hi);
                    } else {
                        part[16 * k + g] = lo;
                        part[16 * k + g + 8] = hi;
                    }
                }
            }
        }
        __syncwarp();
        walk.step(a, p.weight);
    }
    copies_wait<0>();
}

template <typename C, int DP, int NT, int SLOTS, int TEAM>
struct Variant {
    using M = Mma<C, DP, NT, SLOTS, TEAM>;
    static cudaError_t launch(const Args &a, cudaStream_t stream) {
        return launch_kernel<attn_mma_kernel<C, DP, NT, SLOTS, TEAM>, M::kSmem, TEAM>(a, stream);
    }
    static int workers() { return M::kBlocks * M::kWorkers; }
    static int unit() { return M::kKeys; }
};

// Calls f with the variant for these sizes. 8 query rows of a warp, 16 of a team of two (8-bit values, which each warp of a team would
// widen for itself, of one warp while the registers allow it), 32 and 64 of a team of four. (16 sequences of up to 8192
// tokens, 4 key heads of 128: 16 rows over bf16 33 us with two warps and 40 with one, over 8 bits 31 and 29; 32 rows
// as two blocks of 16 instead of a team's 63 and 41, 43 and 42; 64 rows as two of 32 68 and 56, 68 and 65. Few rows in an
// item of 16: 64 sequences over an 8-bit cache 212 us, and 188 in items of 8.)
// Slots of the rings, with one less and one more (us; one token of 16 sequences of 16384, 32768 or 8192 tokens for 128, 64 and 256 channels,
// new tokens over up to 8192, 4 key heads): one less leaves a worker waiting, one more can cost a block of the SM.
//   64 channels:  8 rows bf16 95 (121, 95), 8 bits 73 (70, 107); 16 rows 24 (25, 24), 24 (24, 28); 32 and 64 rows within 2 %
//   128 channels: 8 rows 92 (92, 92), 55 (54, 55); 16 rows 33 (35, 34), 29 (35, 29); 32 rows 42 (39, 41), 41 (41, 42); 64 rows 52 (52, 56), 56 (59, 60)
//   256 channels: 8 rows 92 (91, 92), 57 (54, 59), but one long sequence over 8 bits 36 (37); 16 rows 55 (53, 56), 39 (-, 41); 32 rows 65 (65, 66),
//                 59 (-, 61); 64 rows 109 (111, 113), 100 (-, 102)
template <typename C, int DP, int SLOTS, int SLOTS_TEAM, typename F>
auto pick_rows(const Args &a, F f) {
    if (a.rows == 8) return f(Variant<C, DP, 1, SLOTS, 1>{});
    if constexpr (DP <= 128) {
        if (a.rows == 64) return f(Variant<C, DP, 2, SLOTS_TEAM, 4>{});
    }
    if (a.rows == 16) {
        if constexpr (DP <= 128 && sizeof(C) == 1)
            return f(Variant<C, DP, 2, SLOTS, 1>{});
        else
            return f(Variant<C, DP, 1, SLOTS_TEAM, 2>{});
    }
    return f(Variant<C, DP, 1, SLOTS_TEAM, 4>{});
}
template <typename C, typename F>
auto pick(const Args &a, F f) {
    if (a.cache.D <= 64) return pick_rows<C, 64, 6, 7>(a, f);
    if (a.cache.D <= 128) return pick_rows<C, 128, 4, sizeof(C) == 1 ? 7 : 5>(a, f);
    return pick_rows<C, 256, 3, sizeof(C) == 1 ? 4 : 5>(a, f);
}

}  // namespace

int mma_rows(int all, int D) { return all <= 8 ? 8 : all <= 16 ? 16 : all <= 32 || D > 128 ? 32 : 64; }

int mma_unit_shift(const Args &a) {
    auto f = [](auto v) { return decltype(v)::unit() == 32 ? 5 : 4; };
    return a.cache.ks != nullptr ? pick<uint8_t>(a, f) : pick<bf16>(a, f);
}
int mma_workers(const Args &a) {
    auto f = [](auto v) { return decltype(v)::workers(); };
    return a.cache.ks != nullptr ? pick<uint8_t>(a, f) : pick<bf16>(a, f);
}
cudaError_t launch_attn_mma(const Args &a, cudaStream_t stream) {
    auto f = [&](auto v) { return decltype(v)::launch(a, stream); };
    return a.cache.ks != nullptr ? pick<uint8_t>(a, f) : pick<bf16>(a, f);
}

}  // namespace attn
}  // namespace kda
