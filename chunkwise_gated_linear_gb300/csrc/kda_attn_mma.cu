// Attention over a paged cache, computed by matrix instructions: bf16 queries, cache bf16 or 8-bit. See attn_common.cuh for
// how the work is cut and how keys and values stream in.
//
// Few query rows meet many keys, so the keys are the long side M of the instructions (m16n8k16) and 8 NT query rows the
// short side N: S^T = K Q^T (16 keys x rows), O^T += V^T P^T (channels x rows). K is read from the ring as it lies, V
// through the transposing load; the accumulator of S^T becomes the operand P^T by a transpose of 8 x 8 blocks
// in registers. A row's statistics are shared by the 8 lanes that hold its keys, but the sum is kept per
// lane and the reference m of the exponentials moves only when some score passes it by 2^8 or more, so that
// most steps exchange nothing between lanes.
//
// 8-bit cache: e4m3 numbers are exact in fp16, so K and V are widened in registers and the products run in fp16
// (one conversion per two numbers; widening to bf16 takes four to five instructions). Q goes to fp16 times a power of two per
// row that puts its largest entry at 2^14: entries down to 2^-28 of it stay exact. The power of two of a key multiplies
// its scores, that of a value its probability: P' = 2^(score + sv - M) with a reference M of its own, between 2^-24 and
// 2^14 in fp16 (11 bits), while the sum l keeps the plain 2^(score - m).
#include "attn_common.cuh"
#include "attn_launch.h"

namespace kda {
namespace attn {
namespace {

constexpr float kGrow = 8.f;  // scores may pass their reference by 2^kGrow before it moves

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

template <typename C, int DP, int NT, int STAGES>
struct Mma {
    static constexpr bool kScaled = sizeof(C) == 1;
    // blocks of 16 keys in a unit: two of 8-bit values, where the registers hold the scores of both beside O^T
    static constexpr int kHalves = kScaled && DP * NT <= 256 ? 2 : 1;
    static constexpr int kKeys = 16 * kHalves;
    using S = Stream<C, DP, kKeys, STAGES>;
    static constexpr int kSteps = DP / 16;  // products of S^T, and blocks of 16 channels of O^T
    // shared memory: rings, the plan, exponent bytes
    static constexpr int kPlan = kWarps * S::kBytes;
    static constexpr int kSc = kPlan + kPlanBytes;
    static constexpr int kSmem = kSc + kWarps * S::kScaleBytes;
    static constexpr int kFit = (228 * 1024) / (kSmem + 1024);
    // registers: O^T and Q^T alone are (4 + 2) kSteps NT of a lane's
    static constexpr int kLive = 6 * kSteps * NT + 90;
    static constexpr int kByRegs = 65536 / (kThreads * (kLive < 96 ? 96 : kLive > 255 ? 255 : kLive));
    static constexpr int kBlocks = kFit < kByRegs ? kFit : kByRegs;
};

template <typename C, int DP, int NT, int STAGES>
__global__ void __launch_bounds__(kThreads, Mma<C, DP, NT, STAGES>::kBlocks) attn_mma_kernel(const __grid_constant__ Args a) {
    using M = Mma<C, DP, NT, STAGES>;
    using S = typename M::S;
    constexpr int kSteps = M::kSteps, kHalves = M::kHalves, kKeys = M::kKeys;
    extern __shared__ __align__(1024) unsigned char mem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    launch_dependents();
    Walk walk = find_walk(a, reinterpret_cast<int64_t *>(mem + M::kPlan));
    if (walk.left <= 0) return;
    unsigned char *own = mem + warp * S::kBytes;
    S st(a, own, mem + M::kSc + warp * S::kScaleBytes, lane, walk);
    const int D = a.cache.D;

    int slot = 0;
    while (walk.left > 0) {
        const Piece p = walk.piece(a);
        // Q^T: row 8 n + g, the lane's channels of each block of 16 in the order in which K's come out of the ring
        uint32_t q[NT][kSteps][2];
        float rowf[NT][2];  // what a score of rows 8 n + 2 c, + 1 is multiplied with
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const bool there = 8 * n + g < p.rows;
            const bf16 *from = static_cast<const bf16 *>(a.q) + (there ? q_at(a, p, 8 * n + g) : 0);
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                q[n][k][0] = q[n][k][1] = 0u;
                if (there && 16 * k < D) {
                    if constexpr (M::kScaled) {
                        const uint2 x = *reinterpret_cast<const uint2 *>(from + 16 * k + 4 * c);
                        q[n][k][0] = x.x;
                        q[n][k][1] = x.y;
                    } else {
                        q[n][k][0] = *reinterpret_cast<const uint32_t *>(from + 16 * k + 2 * c);
                        q[n][k][1] = *reinterpret_cast<const uint32_t *>(from + 16 * k + 2 * c + 8);
                    }
                }
            }
            if constexpr (M::kScaled) {
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        top = fmaxf(top, finite_abs(__uint_as_float(q[n][k][i] << 16)));
                        top = fmaxf(top, finite_abs(__uint_as_float(q[n][k][i] & 0xffff0000u)));
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // 2^e with the largest entry at 2^14 .. 2^15, within what fp32 holds
                int e = 127 + 14 - (int)(__float_as_uint(top) >> 23);
                e = e > 126 ? 126 : e;
                const float up = pow2(e);
#pragma unroll
                for (int k = 0; k < kSteps; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        q[n][k][i] = pack_f16(__uint_as_float(q[n][k][i] << 16) * up, __uint_as_float(q[n][k][i] & 0xffff0000u) * up);
                const float down = a.scale_log2 * pow2(-e);
#pragma unroll
                for (int j = 0; j < 2; ++j) rowf[n][j] = __shfl_sync(0xffffffffu, down, 4 * (2 * c + j));
            } else {
                rowf[n][0] = rowf[n][1] = a.scale_log2;
            }
        }
        const int least = seen(a, p.len, p.row0);  // keys from here on are not seen by all rows

        float o[kSteps][NT][4];
        float m[NT][2], l[NT][2], big[NT][2];  // reference of the exponentials, their sum, where the reference moves
        float mv[NT][2], bigv[NT][2];          // 8-bit: the reference M of P', where it moves
        float turn[NT][2];                     // 8-bit: 2^(m - M)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m[n][j] = mv[n][j] = l[n][j] = 0.f;
                turn[n][j] = 1.f;
                big[n][j] = bigv[n][j] = -INFINITY;
            }
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[k][n][i] = 0.f;
        }

        for (int u = p.u0; u < p.u1; ++u) {
            st.ready();
            const int pos0 = u * kKeys;
            if (pos0 < p.last) {  // the same for the whole warp
                const uint32_t ks = st.ring + slot * 2 * S::kHalf, vs = ks + S::kHalf;
                // scores, base 2; element i of half h: key 16 h + g + 8 (i / 2), row 8 n + 2 c + i % 2
                float x[kHalves][NT][4];
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[h][n][i] = 0.f;
                const uint32_t krow = ks + (lane & 15) * S::kPitch;
#pragma unroll
                for (int k = 0; k < kSteps; k += M::kScaled ? 2 : 1) {
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) {
                        uint32_t r[4];
                        if constexpr (M::kScaled) {
                            // 16-byte chunks k and k + 1 are channels 16 k .. 16 k + 31: keys g and g + 8, channels 4 c .. 4 c + 3 of each
                            ldsm(r, krow + 16 * h * S::kPitch + (((k + (lane >> 4)) ^ (lane & 7)) << 4));
                            uint32_t f[4];
                            widen(r[0], f[0], f[2]);
                            widen(r[1], f[1], f[3]);
#pragma unroll
                            for (int n = 0; n < NT; ++n) mma_f16(x[h][n], f, q[n][k][0], q[n][k][1]);
                            widen(r[2], f[0], f[2]);
                            widen(r[3], f[1], f[3]);
#pragma unroll
                            for (int n = 0; n < NT; ++n) mma_f16(x[h][n], f, q[n][k + 1][0], q[n][k + 1][1]);
                        } else {
                            ldsm(r, krow + 16 * h * S::kPitch + (((2 * k + (lane >> 4)) ^ (lane & 7)) << 4));
#pragma unroll
                            for (int n = 0; n < NT; ++n) mma_bf16(x[h][n], r, q[n][k][0], q[n][k][1]);
                        }
                    }
                }
                float fv[kHalves][2], ev[kHalves][2];  // 8-bit: the values' powers of two and their exponents
                const bool edge = pos0 + kKeys > least;
                bool grows = false;
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    float fk[2] = {1.f, 1.f};
                    if constexpr (M::kScaled) {
                        const uint8_t *sc = st.scales + slot * 2 * kKeys + 16 * h;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            fk[i] = __uint_as_float((uint32_t)sc[g + 8 * i] << 23);
                            const uint32_t e = sc[kKeys + g + 8 * i];
                            fv[h][i] = __uint_as_float(e << 23);
                            ev[h][i] = (float)((int)e - 127);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float &y = x[h][n][i];
                            y *= M::kScaled ? rowf[n][i & 1] * fk[i >> 1] : rowf[n][i & 1];
                            if (edge && pos0 + 16 * h + g + 8 * (i >> 1) >= seen(a, p.len, p.row0 + 8 * n + 2 * c + (i & 1))) y = -INFINITY;
                            grows |= y > big[n][i & 1];
                            if constexpr (M::kScaled) grows |= y + ev[h][i >> 1] > bigv[n][i & 1];
                        }
                }
                if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float top = -INFINITY, topv = -INFINITY;
#pragma unroll
                            for (int h = 0; h < kHalves; ++h)
#pragma unroll
                                for (int i = j; i < 4; i += 2) {
                                    top = fmaxf(top, x[h][n][i]);
                                    if constexpr (M::kScaled) topv = fmaxf(topv, x[h][n][i] + ev[h][i >> 1]);
                                }
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) {
                                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                                if constexpr (M::kScaled) topv = fmaxf(topv, __shfl_xor_sync(0xffffffffu, topv, d));
                            }
                            // each reference moves up alone, never down; nothing seen yet: l and O are 0
                            float back = 1.f;
                            if (top > big[n][j] - kGrow) {
                                back = big[n][j] == -INFINITY ? 0.f : tc5::ex2(m[n][j] - top);
                                l[n][j] *= back;
                                m[n][j] = top;
                                big[n][j] = top + kGrow;
                            }
                            if constexpr (M::kScaled) {
                                // the largest P' at 2^6, so that none passes 2^14; rows of zeros (sv = -126) alone leave it lower,
                                // or 2^(m - M) would pass what fp32 holds
                                const float tv = fmaxf(topv, bigv[n][j] - kGrow);
                                const float to = fmaxf(tv - 6.f, m[n][j] - 120.f);
                                back = 1.f;
                                if (tv > -INFINITY) {
                                    back = bigv[n][j] == -INFINITY ? 0.f : tc5::ex2(mv[n][j] - to);
                                    mv[n][j] = to;
                                    bigv[n][j] = tv + kGrow;
                                }
                                turn[n][j] = tc5::ex2(m[n][j] - mv[n][j]);
                            }
                            if (back != 1.f) {
#pragma unroll
                                for (int k = 0; k < kSteps; ++k) {
                                    o[k][n][j] *= back;
                                    o[k][n][j + 2] *= back;
                                }
                            }
                        }
                }
                uint32_t pb[kHalves][NT][2];
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float &y = x[h][n][i];
                            y = tc5::ex2(y - m[n][i & 1]);
                            l[n][i & 1] += y;
                            if constexpr (M::kScaled) y *= fv[h][i >> 1] * turn[n][i & 1];
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float lo = x[h][n][2 * i], hi = x[h][n][2 * i + 1];
                            pb[h][n][i] = transpose8(M::kScaled ? pack_f16(lo, hi) : pack_bf16(lo, hi));
                        }
                    }
                if (edge && a.T > 1) {
                    // Values that are not finite would reach rows that do not see them, as 0 * NaN: such keys' shares are added one by
                    // one to the rows that do, and their values then count as zeros.
                    unsigned char *vals = own + slot * 2 * S::kHalf + S::kHalf;
                    uint32_t odd = 0;
                    for (int r = 0; r < kKeys; ++r) {
                        bool bad = false;
                        for (int w = lane; w < S::kPitch / 4; w += 32) {
                            const uint32_t v = *reinterpret_cast<const uint32_t *>(vals + r * S::kPitch + 4 * w);
                            if constexpr (M::kScaled)
                                bad |= (v & 0x7fu) == 0x7fu || (v >> 8 & 0x7fu) == 0x7fu || (v >> 16 & 0x7fu) == 0x7fu || (v >> 24 & 0x7fu) == 0x7fu;
                            else
                                bad |= (v & 0x7f80u) == 0x7f80u || (v >> 16 & 0x7f80u) == 0x7f80u;
                        }
                        if (__any_sync(0xffffffffu, bad)) odd |= 1u << r;
                    }
                    if (odd != 0) {
#pragma unroll
                        for (int h = 0; h < kHalves; ++h)
#pragma unroll 1
                            for (int r = 0; r < 16; ++r) {
                                if ((odd >> (16 * h + r) & 1) == 0) continue;
#pragma unroll
                                for (int n = 0; n < NT; ++n)
#pragma unroll
                                    for (int j = 0; j < 2; ++j) {
                                        const float lo = __shfl_sync(0xffffffffu, x[h][n][j], 4 * (r & 7) + c);
                                        const float hi = __shfl_sync(0xffffffffu, x[h][n][j + 2], 4 * (r & 7) + c);
                                        const float w = r < 8 ? lo : hi;
                                        if (pos0 + 16 * h + r >= seen(a, p.len, p.row0 + 8 * n + 2 * c + j)) continue;
#pragma unroll
                                        for (int k = 0; k < kSteps; ++k)
#pragma unroll
                                            for (int t = 0; t < 2; ++t) {
                                                const int byte = (16 * k + (M::kScaled ? 2 * g + t : g + 8 * t)) * (int)sizeof(C);
                                                const unsigned char *e = vals + (16 * h + r) * S::kPitch + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15);
                                                float v, no;
                                                if constexpr (M::kScaled)
                                                    e4m3_to_f(*e, v, no);
                                                else
                                                    v = to_f(*reinterpret_cast<const bf16 *>(e));
                                                o[k][n][j + 2 * t] = fmaf(w, v, o[k][n][j + 2 * t]);
                                            }
                                    }
                            }
                        __syncwarp();
                        for (int r = 0; r < kKeys; ++r)
                            if (odd >> r & 1)
                                for (int w = lane; w < S::kPitch / 4; w += 32) *reinterpret_cast<uint32_t *>(vals + r * S::kPitch + 4 * w) = 0u;
                        __syncwarp();
                    }
                }
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    if constexpr (M::kScaled) {
                        // 16 keys x 16-byte chunks k, k + 1, transposed in units of two bytes: channels 2 g, 2 g + 1 of keys 2 c, 2 c + 1
                        const uint32_t vrow = vs + (16 * h + (lane & 15)) * S::kPitch;
#pragma unroll
                        for (int k = 0; k < kSteps; k += 2) {
                            uint32_t r[4];
                            ldsm_t(r, vrow + (((k + (lane >> 4)) ^ (lane & 7)) << 4));
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                // bytes (key 2c, channel 2g), (2c, 2g + 1), (2c + 1, 2g), (2c + 1, 2g + 1): pair the keys
                                uint32_t f[4];
                                widen(__byte_perm(r[2 * t], 0, 0x3120), f[0], f[1]);
                                widen(__byte_perm(r[2 * t + 1], 0, 0x3120), f[2], f[3]);
#pragma unroll
                                for (int n = 0; n < NT; ++n) mma_f16(o[k + t][n], f, pb[h][n][0], pb[h][n][1]);
                            }
                        }
                    } else {
                        const uint32_t vrow = vs + (16 * h + (lane & 7) + ((lane >> 4) << 3)) * S::kPitch;
#pragma unroll
                        for (int k = 0; k < kSteps; ++k) {
                            uint32_t r[4];
                            ldsm_t(r, vrow + (((2 * k + ((lane >> 3) & 1)) ^ (lane & 7)) << 4));
#pragma unroll
                            for (int n = 0; n < NT; ++n) mma_bf16(o[k][n], r, pb[h][n][0], pb[h][n][1]);
                        }
                    }
                }
            }
            slot = st.next(slot);
        }
        float *piece = piece_mem(a, blockIdx.x * kWarps + warp, p.u0 == 0);
        const bool whole = p.whole();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], d);
                const int r = 8 * n + 2 * c + j;
                if (r >= p.rows) continue;
                const float top = big[n][j] == -INFINITY ? -INFINITY : m[n][j];
                float f = M::kScaled ? tc5::ex2(mv[n][j] - m[n][j]) : 1.f;
                if (whole) {
                    f = l[n][j] == 0.f ? 0.f : f / l[n][j];
                    const int64_t row = out_row(a, p, r);
                    bf16 *to = static_cast<bf16 *>(a.o) + row * D;
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        if (16 * k >= D) break;
                        const float lo = o[k][n][j] * f, hi = o[k][n][j + 2] * f;
                        if constexpr (M::kScaled) {
                            *reinterpret_cast<uint32_t *>(to + 16 * k + 2 * g) = pack_bf16(lo, hi);
                        } else {
                            to[16 * k + g] = from_f<bf16>(lo);
                            to[16 * k + g + 8] = from_f<bf16>(hi);
                        }
                    }
                    if (g == 0 && a.lse != nullptr) a.lse[row] = lse_of(top, l[n][j]);
                } else {
                    float *to = piece + r * D;
#pragma unroll
                    for (int k = 0; k < kSteps; ++k) {
                        if (16 * k >= D) break;
                        const float lo = o[k][n][j] * f, hi = o[k][n][j + 2] * f;
                        if constexpr (M::kScaled) {
                            *reinterpret_cast<float2 *>(to + 16 * k + 2 * g) = make_float2(lo, hi);
                        } else {
                            to[16 * k + g] = lo;
                            to[16 * k + g + 8] = hi;
                        }
                    }
                    if (g == 0) reinterpret_cast<float2 *>(piece + a.rows * D)[r] = make_float2(top, l[n][j]);
                }
            }
        }
        walk.step(a, p);
    }
    copies_wait<0>();
}

template <typename C, int DP, int NT, int STAGES>
struct Variant {
    using M = Mma<C, DP, NT, STAGES>;
    static cudaError_t launch(const Args &a, cudaStream_t stream) {
        return launch_kernel<attn_mma_kernel<C, DP, NT, STAGES>, M::kSmem>(a, stream);
    }
    static int blocks() { return M::kBlocks; }
    static int unit() { return M::kKeys; }
};

// Calls f with the variant for these sizes. Query rows: 8, 16 or 32 (16 where O^T of wide heads fills the registers).
template <typename C, typename F>
auto pick(const Args &a, F f) {
    if (a.cache.D <= 64)
        return a.rows == 8 ? f(Variant<C, 64, 1, 4>{}) : a.rows == 16 ? f(Variant<C, 64, 2, 4>{}) : f(Variant<C, 64, 4, 4>{});
    if (a.cache.D <= 128)
        return a.rows == 8 ? f(Variant<C, 128, 1, 3>{}) : a.rows == 16 ? f(Variant<C, 128, 2, 3>{}) : f(Variant<C, 128, 4, sizeof(C) == 1 ? 6 : 3>{});
    return a.rows == 8 ? f(Variant<C, 256, 1, 3>{}) : f(Variant<C, 256, 2, 3>{});
}

}  // namespace

int mma_rows(int all, int D) { return all <= 8 ? 8 : (all <= 16 || D > 128) ? 16 : 32; }

int mma_unit(const Args &a) {
    auto f = [](auto v) { return decltype(v)::unit(); };
    return a.cache.ks != nullptr ? pick<uint8_t>(a, f) : pick<bf16>(a, f);
}
int mma_blocks(const Args &a) {
    auto f = [](auto v) { return decltype(v)::blocks(); };
    return a.cache.ks != nullptr ? pick<uint8_t>(a, f) : pick<bf16>(a, f);
}
cudaError_t launch_attn_mma(const Args &a, cudaStream_t stream) {
    auto f = [&](auto v) { return decltype(v)::launch(a, stream); };
    return a.cache.ks != nullptr ? pick<uint8_t>(a, f) : pick<bf16>(a, f);
}

}  // namespace attn
}  // namespace kda
