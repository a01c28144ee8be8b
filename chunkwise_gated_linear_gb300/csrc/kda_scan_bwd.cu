// Gradient of the selective state space scan (kda_mixer.h: kda_scan_bwd).
//
// With a_t = exp(delta_t A), x_t = delta_t u_t, g_t = dy_t silu(z_t) and the adjoint
//   l_t = C_t g_t + G_t,   G_t = a_{t+1} l_{t+1}  (dht at a sequence's last token),
// per channel (n runs over the states):
//   s_t = sum_n l_t B_t            du_t = D g_t + delta_t s_t
//   w_t = sum_n A l_t a_t h_{t-1}  ddelta_t = w_t + u_t s_t,  ddt_t = ddelta_t sigmoid(dt_t + bias)
//   y_t = sum_n C_t h_t            dz_t = dy_t (y_t + D u_t) silu'(z_t)
//   dA = sum_t delta_t l_t a_t h_{t-1},   dh0 = a_0 l_0
//   dB_t = sum_d l_t x_t,  dC_t = sum_d g_t h_t   over the channels of a group.
// The states are needed backwards and cannot be undone (a_t may underflow), so they are computed
// again in three steps:
//   1. scan_bwd_local_kernel: the rows are cut into chunks, all walked at once from a zero state.
//      It leaves the local state at every 32 rows (a window), the chunk's end state, its adjoint
//      at the start from a zero adjoint at the end (in the same forward walk:
//      sum_t (a_c0 .. a_t) C_t g_t), and sums of delta.
//   2. scan_bwd_carry_kernel: true states at the chunk starts, true adjoints at the ends.
//   3. scan_bwd_kernel: per chunk and 64 channels, windows last to first. A window's start state
//      is its local state plus exp(A sum delta) times the chunk's start state; from there the
//      states at every fourth token go to shared memory, and groups of four tokens are taken last to first:
//      a and a h_{t-1} of four tokens in registers, then backwards.
// Sums over the states go across 4 lanes, sums over channels across 8 lanes (one exchange per
// value and halving, so that each lane ends with one total), then over warps and blocks in a
// fixed order. About 20 instructions per (token, channel, state): bound by issue.
#include "scan_common.cuh"

namespace kda {
namespace scan {

namespace {

constexpr int kWin = 32;        // tokens per window
constexpr int kGroups = kWin / 4;
constexpr float kLn2 = 0.6931471805599453f;

struct BwdArgs {
    ScanArgs f;         // hchunk: [nchunks][ch][N] end states, then start states; schunk [nchunks][ch]
    const void *dy;
    const float *dht;
    void *du, *ddt, *dB, *dC, *dz;
    float *dh0;
    float *gchunk;      // [nchunks][ch][N]: local start adjoints, then the adjoint that enters at the end
    float *hwin;        // [windows][ch][N]: local states before a window
    float *swin;        // [windows][ch]: sum of delta from the chunk's start to the window
    float *pbc;         // [blocks_per_group][rows][G][2][N]: dB and dC of 64 channels
    float *partial;     // [nchunks][ch N + 2 ch]: dA, dD, ddt_bias
};

// ---- 1: every chunk from zero ---------------------------------------------------------------
// As the forward kernel: a thread owns its channel's states (NS of them, LN lanes per channel), B and C come
// from shared memory, the rest from memory four tokens ahead. One channel per thread: a second one
// would need 128 registers for states, decays, products and adjoints alone.
constexpr int kLThr = 128;
template <typename T, int NS, int LN>
__global__ void __launch_bounds__(kLThr, 4) scan_bwd_local_kernel(const BwdArgs b) {
    constexpr int kNT = NS * LN, P2 = NS / 2, kChan = kLThr / LN;
    constexpr int kBC = 2 * kWin * kNT / kLThr;
    __shared__ __align__(16) float sB[kWin * kNT], sC[kWin * kNT];
    const ScanArgs &a = b.f;
    const int tid = threadIdx.x;
    const int nblk = a.G * a.blocks_per_group;
    const int blk = blockIdx.x % nblk;
    const int64_t part = blockIdx.x / nblk;
    const int g = blk / a.blocks_per_group;
    const int first = (blk % a.blocks_per_group) * kChan + tid / LN;
    const int n0 = (tid % LN) * NS;
    const bool live = first < a.chg;
    const int d = g * a.chg + (live ? first : 0);
    const int64_t cn = (int64_t)a.ch * a.N, dn = (int64_t)d * a.N;
    const bool vst = a.vec_states && a.N == kNT;
    const int64_t c0 = part * a.chunk;
    const int64_t c1 = c0 + a.chunk < a.seqs.rows ? c0 + a.chunk : a.seqs.rows;
    if (c0 >= c1) return;
    SeqAt at = seq_find(a.seqs, c0);

    f2 h[P2], A2[P2], P[P2], f[P2];
    get_states<NS>(h, a.h0, at.s * cn + dn, n0, a.N, live && c0 == at.start && a.h0 != nullptr, vst);
    get_states<NS>(A2, a.A, dn, n0, a.N, live, vst);
#pragma unroll
    for (int i = 0; i < P2; ++i) {
        A2[i] = mul2(A2[i], pk(kLog2e, kLog2e));
        P[i] = pk(1.f, 1.f);
        f[i] = 0;
    }
    float S = 0.f;
    // the adjoint from the end of a sequence: dht, through the decays since the chunk's start
    auto add_dht = [&]() {
        if (b.dht == nullptr) return;
        f2 t[P2];
        get_states<NS>(t, b.dht, at.s * cn + dn, n0, a.N, live, vst);
#pragma unroll
        for (int i = 0; i < P2; ++i) f[i] = fma2(P[i], t[i], f[i]);
    };
    const float bias = a.bias != nullptr ? a.bias[d] : 0.f;
    const bool gate = a.z != nullptr;

    T nu[4], ndt[4], ndy[4], nz[4];
    auto fetch = [&](int64_t r0) {
        const T *pu = static_cast<const T *>(a.u) + r0 * a.us, *pd = static_cast<const T *>(a.dt) + r0 * a.dts;
        const T *py = static_cast<const T *>(b.dy) + r0 * a.ch, *pz = static_cast<const T *>(a.z) + r0 * a.zs;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (r0 + k < c1) {
                nu[k] = pu[k * a.us + d];
                ndt[k] = pd[k * a.dts + d];
                ndy[k] = py[(int64_t)k * a.ch + d];
                if (gate) nz[k] = pz[k * a.zs + d];
            }
    };
    float nbc[kBC];
    auto fetch_bc = [&](int64_t t0) {
#pragma unroll
        for (int k = 0; k < kBC; ++k) {
            const bool isC = k >= kBC / 2;
            const int e = (tid + k * kLThr) % (kWin * kNT);
            const int64_t r = t0 + e / kNT;
            const int n = e % kNT;
            nbc[k] = r < c1 && n < a.N
                         ? to_f(static_cast<const T *>(isC ? a.C : a.B)[r * (isC ? a.cs : a.bs) + (int64_t)g * a.N + n])
                         : 0.f;
        }
    };
    auto token = [&](int t, T ru, T rdt, T rdy, T rz) {
        const float delta = step_of<T>(to_f(rdt) + bias, a.softplus), x = delta * to_f(ru);
        const float gy = gate ? to_f(rdy) * act_value(to_f(rz), true) : to_f(rdy);
        const f2 d2 = pk(delta, delta), x2 = pk(x, x), g2 = pk(gy, gy);
        S += delta;
#pragma unroll
        for (int i = 0; i < P2; i += 2) {
            const ulonglong2 B = *reinterpret_cast<const ulonglong2 *>(&sB[t * kNT + n0 + 2 * i]);
            const ulonglong2 C = *reinterpret_cast<const ulonglong2 *>(&sC[t * kNT + n0 + 2 * i]);
            const f2 e0 = exp2_2(mul2(d2, A2[i])), e1 = exp2_2(mul2(d2, A2[i + 1]));
            h[i] = fma2(e0, h[i], mul2(x2, B.x));
            h[i + 1] = fma2(e1, h[i + 1], mul2(x2, B.y));
            P[i] = mul2(P[i], e0);
            P[i + 1] = mul2(P[i + 1], e1);
            f[i] = fma2(P[i], mul2(g2, C.x), f[i]);
            f[i + 1] = fma2(P[i + 1], mul2(g2, C.y), f[i + 1]);
        }
    };
    fetch(c0);
    fetch_bc(c0);
    for (int64_t t0 = c0; t0 < c1; t0 += kWin) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kBC; ++k) (k < kBC / 2 ? sB : sC)[(tid + k * kLThr) % (kWin * kNT)] = nbc[k];
        __syncthreads();
        if (t0 + kWin < c1) fetch_bc(t0 + kWin);
        if (t0 > c0) {  // the state before this window
            put_states<NS>(h, b.hwin, (t0 / kWin) * cn + dn, n0, a.N, live, a.N == kNT);
            if (live && n0 == 0) b.swin[(t0 / kWin) * a.ch + d] = S;
        }
#pragma unroll 1
        for (int t = 0; t < kWin; t += 4) {
            const int64_t r = t0 + t;
            if (r >= c1) break;
            T cu_[4], cdt[4], cdy[4], cz[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                cu_[k] = nu[k];
                cdt[k] = ndt[k];
                cdy[k] = ndy[k];
                cz[k] = nz[k];
            }
            if (r + 4 < c1) fetch(r + 4);
            if (r + 4 <= c1 && r + 4 <= at.end) {
#pragma unroll
                for (int k = 0; k < 4; ++k) token(t + k, cu_[k], cdt[k], cdy[k], cz[k]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (r + k >= c1) break;
                    if (r + k == at.end) {
                        add_dht();
#pragma unroll
                        for (int i = 0; i < P2; ++i) P[i] = 0;
                        seq_next(a.seqs, at);
                        get_states<NS>(h, a.h0, at.s * cn + dn, n0, a.N, live && a.h0 != nullptr, vst);
                    }
                    token(t + k, cu_[k], cdt[k], cdy[k], cz[k]);
                }
            }
        }
    }
    if (c1 == at.end) add_dht();
    put_states<NS>(h, a.hchunk, part * cn + dn, n0, a.N, live, a.N == kNT);
    put_states<NS>(f, b.gchunk, part * cn + dn, n0, a.N, live, a.N == kNT);
    if (live && n0 == 0) a.schunk[part * a.ch + d] = S;
}

template <typename T, int NS, int LN>
cudaError_t launch_local(BwdArgs b, cudaStream_t stream) {
    b.f.blocks_per_group = (int)ceil_div(b.f.chg, kLThr / LN);
    const int64_t grid = b.f.nchunks * b.f.G * b.f.blocks_per_group;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    scan_bwd_local_kernel<T, NS, LN><<<(unsigned)grid, kLThr, 0, stream>>>(b);
    return cudaGetLastError();
}

// ---- 2: between the chunks, in place ----------------------------------------------------------
// Adjoints (states: scan_carry_kernel): the adjoint that enters chunk c - 1 at its end is chunk
// c's local one plus, when no sequence ends in chunk c, exp(A sum delta) times what enters c.
__global__ void __launch_bounds__(256) scan_bwd_carry_kernel(const BwdArgs b) {
    const ScanArgs &a = b.f;
    constexpr int kAhead = 8;
    __shared__ bool ends[256];
    const int64_t total = (int64_t)a.ch * a.N;
    const int64_t at_e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t e = at_e < total ? at_e : total - 1;
    const int d = (int)(e / a.N);
    const float A = a.A[e] * kLog2e;
    float in = 0.f;
    for (int64_t k = 0; k < a.nchunks; k += kAhead) {  // k counts chunks from the last
        if (k % 256 == 0) {
            __syncthreads();
            const int64_t c = a.nchunks - 1 - (k + threadIdx.x);
            const int64_t c0 = c * a.chunk, c1 = c0 + a.chunk;
            ends[threadIdx.x] = c < 0 || c1 >= a.seqs.rows || seq_find(a.seqs, c0).end <= c1;
            __syncthreads();
        }
        float loc[kAhead], sum[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t c = a.nchunks - 1 - (k + i);
            if (c > 0) {
                loc[i] = b.gchunk[c * total + e];
                sum[i] = a.schunk[c * a.ch + d];
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t c = a.nchunks - 1 - (k + i);
            if (c < 0) break;
            if (at_e < total) b.gchunk[c * total + e] = in;
            if (c > 0) in = ends[(k + i) % 256] ? loc[i] : fmaf(tc5::ex2(A * sum[i]), in, loc[i]);
        }
    }
}

// ---- 3: the gradients -------------------------------------------------------------------------
// Sums of eight values over the eight lanes that differ in bits 2..4: lane l gets the total of
// value l / 4.
__device__ __forceinline__ float sum_channels(const float (&v)[8], int lane) {
    const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
    float w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float s = b4 ? v[j] : v[j + 4], k = b4 ? v[j + 4] : v[j];
        w[j] = k + __shfl_xor_sync(0xffffffffu, s, 16);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float s = b3 ? w[j] : w[j + 2], k = b3 ? w[j + 2] : w[j];
        w[j] = k + __shfl_xor_sync(0xffffffffu, s, 8);
    }
    const float s = b2 ? w[0] : w[1], k = b2 ? w[1] : w[0];
    return k + __shfl_xor_sync(0xffffffffu, s, 4);
}

// R channels per thread: two while their states are few (half the exchanges per state).
template <int NP>
struct BwdShape {
    static constexpr int R = NP <= 4 ? 2 : 1;
    static constexpr int E = R * NP;               // states per thread
    static constexpr int kThr = kDB * kLN / R;
    static constexpr int kWarps = kThr / 32;
    static constexpr int kNT = kLN * NP;
    static constexpr int kCkpt = kGroups * E * kThr * 4;  // states at every fourth token
    static constexpr int kTile = kWin * kDB * 16;         // delta, x, g; then s, w, y
    static constexpr int kBCBytes = 2 * kWin * kNT * 4;
    static constexpr int kFlags = kWin * 8;               // per row: sequence, start / end bits
    static constexpr int kSmem = kCkpt + kTile + kBCBytes + kFlags;
};

template <typename T, int NP>
struct BwdBlock {
    using S = BwdShape<NP>;
    static constexpr int R = S::R, P2 = NP / 2;
    const BwdArgs &b;
    float4 *tile;        // [kWin][kDB]
    const float *sB, *sC;
    float4 *ckpt;        // [kGroups][kWarps][E / 4][32]
    const int *seq_of, *flag_of;
    int lane, warp, nl;
    int dl[R];           // the thread's channels in the block
    int64_t dn[R];       // and their place in [ch][N]
    bool live[R];
    f2 A2[R][P2], G[R][P2], dA[R][P2];

    __device__ __forceinline__ BwdBlock(const BwdArgs &args) : b(args) {}
    __device__ __forceinline__ float *group_mem(int g) const {
        return reinterpret_cast<float *>(ckpt + (g * S::kWarps + warp) * (S::E / 4) * 32);
    }
    __device__ __forceinline__ void state_of(f2 (&h)[R][P2], const float *base, int s) const {
        const ScanArgs &a = b.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float t[NP];
            load_states<NP>(t, base, s * (int64_t)a.ch * a.N + dn[r], nl, a.N, live[r] && base != nullptr);
            to_pairs<NP>(h[r], t);
        }
    }
    // states before tokens 0, 4, .. of the window into shared memory, from the state h before it
    template <bool RAG>
    __device__ __forceinline__ void forward(f2 (&h)[R][P2]) const {
        for (int g = 0; g < kGroups; ++g) {
            float4 *to = reinterpret_cast<float4 *>(group_mem(g));
#pragma unroll
            for (int q = 0; q < S::E / 4; ++q) {
                const f2 lo = h[(4 * q) / NP][((4 * q) % NP) / 2], hi = h[(4 * q + 2) / NP][((4 * q + 2) % NP) / 2];
                float4 v;
                upk(lo, v.x, v.y);
                upk(hi, v.z, v.w);
                to[q * 32 + lane] = v;
            }
            if (g == kGroups - 1) break;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = 4 * g + k;
                if (RAG && (flag_of[t] & 1)) state_of(h, b.f.h0, seq_of[t]);
                f2 B[P2];
                lds_pairs<NP>(B, sB + t * S::kNT + nl * NP);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float2 dx = *reinterpret_cast<const float2 *>(&tile[t * kDB + slot_of(dl[r])]);
                    const f2 d2 = pk(dx.x, dx.x), x2 = pk(dx.y, dx.y);
#pragma unroll
                    for (int i = 0; i < P2; ++i) h[r][i] = fma2(exp2_2(mul2(d2, A2[r][i])), h[r][i], mul2(x2, B[i]));
                }
            }
        }
    }
    // tokens 4 g + 3 .. 4 g of the window
    template <bool RAG>
    __device__ __forceinline__ void backward(int g) {
        float *mem = group_mem(g);
        f2 h[R][P2], e[4][R][P2], eh[4][R][P2];
        float dlt[4][R], x[4][R], gr[4][R];
#pragma unroll
        for (int q = 0; q < S::E / 4; ++q) {
            const float4 v = reinterpret_cast<const float4 *>(mem)[q * 32 + lane];
            h[(4 * q) / NP][((4 * q) % NP) / 2] = pk(v.x, v.y);
            h[(4 * q + 2) / NP][((4 * q + 2) % NP) / 2] = pk(v.z, v.w);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int t = 4 * g + k;
            if (RAG && (flag_of[t] & 1)) state_of(h, b.f.h0, seq_of[t]);
            f2 B[P2];
            lds_pairs<NP>(B, sB + t * S::kNT + nl * NP);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float4 q = tile[t * kDB + slot_of(dl[r])];
                dlt[k][r] = q.x;
                x[k][r] = q.y;
                gr[k][r] = q.z;
                const f2 d2 = pk(q.x, q.x), x2 = pk(q.y, q.y);
#pragma unroll
                for (int i = 0; i < P2; ++i) {
                    e[k][r][i] = exp2_2(mul2(d2, A2[r][i]));
                    eh[k][r][i] = mul2(e[k][r][i], h[r][i]);
                    h[r][i] = fma2(x2, B[i], eh[k][r][i]);
                }
            }
        }
        __syncwarp();  // the group's states have been read: its memory takes dB and dC
        float s[R][4], w[R][4], y[R][4];
#pragma unroll
        for (int k = 3; k >= 0; --k) {
            const int t = 4 * g + k;
            if (RAG && (flag_of[t] & 2)) state_of(G, b.dht, seq_of[t]);
            f2 B[P2], C[P2], dB[P2], dC[P2];
            lds_pairs<NP>(B, sB + t * S::kNT + nl * NP);
            lds_pairs<NP>(C, sC + t * S::kNT + nl * NP);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const f2 d2 = pk(dlt[k][r], dlt[k][r]), x2 = pk(x[k][r], x[k][r]), g2 = pk(gr[k][r], gr[k][r]);
                f2 s2 = 0, w2 = 0, y2 = 0;
#pragma unroll
                for (int i = 0; i < P2; ++i) {
                    const f2 l = fma2(g2, C[i], G[r][i]);
                    const f2 ht = fma2(x2, B[i], eh[k][r][i]);
                    const f2 q = mul2(l, eh[k][r][i]);
                    dB[i] = r == 0 ? mul2(l, x2) : fma2(l, x2, dB[i]);
                    dC[i] = r == 0 ? mul2(ht, g2) : fma2(ht, g2, dC[i]);
                    s2 = i == 0 ? mul2(l, B[i]) : fma2(l, B[i], s2);
                    y2 = i == 0 ? mul2(ht, C[i]) : fma2(ht, C[i], y2);
                    w2 = i == 0 ? mul2(q, A2[r][i]) : fma2(q, A2[r][i], w2);
                    dA[r][i] = fma2(q, d2, dA[r][i]);
                    G[r][i] = mul2(l, e[k][r][i]);
                }
                s[r][k] = hsum2(s2);
                w[r][k] = hsum2(w2);
                y[r][k] = hsum2(y2);
            }
            if (RAG && (flag_of[t] & 1) && b.dh0 != nullptr) {
                const ScanArgs &a = b.f;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float o[NP];
                    from_pairs<NP>(o, G[r]);
                    store_states<NP>(o, b.dh0, seq_of[t] * (int64_t)a.ch * a.N + dn[r], nl, a.N, live[r]);
                }
            }
            // [which][4 NP] of token t, this warp's channels added up
            float vb[NP], vc[NP];
            from_pairs<NP>(vb, dB);
            from_pairs<NP>(vc, dC);
            float *to = mem + k * 2 * S::kNT;
            const int j = lane >> 2;
            if constexpr (NP >= 8) {
#pragma unroll
                for (int q = 0; q < NP / 8; ++q) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = vb[8 * q + i];
                    to[nl * NP + 8 * q + j] = sum_channels(v, lane);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = vc[8 * q + i];
                    to[S::kNT + nl * NP + 8 * q + j] = sum_channels(v, lane);
                }
            } else {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = i < NP ? vb[i % NP] : (i < 2 * NP ? vc[i % NP] : 0.f);
                const float tot = sum_channels(v, lane);
                if (j < 2 * NP) to[(j / NP) * S::kNT + nl * NP + j % NP] = tot;
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float s1 = sum_lanes(s[r], nl), w1 = sum_lanes(w[r], nl), y1 = sum_lanes(y[r], nl);
            __syncwarp();
            tile[(4 * g + nl) * kDB + slot_of(dl[r])] = make_float4(s1, w1 * kLn2, y1, 0.f);
        }
    }
};

template <typename T, int NP>
__global__ void __launch_bounds__(BwdShape<NP>::kThr) scan_bwd_kernel(const BwdArgs b) {
    using S = BwdShape<NP>;
    constexpr int R = S::R, P2 = NP / 2, kThr = S::kThr;
    constexpr int kRowsAt = kThr / 8;  // token rows staged at a time
    extern __shared__ __align__(16) unsigned char smem[];
    const ScanArgs &a = b.f;
    const int tid = threadIdx.x;
    const int nblk = a.G * a.blocks_per_group;
    const int blk = blockIdx.x % nblk;
    const Chans ch = chans_of(a, blk);
    const int64_t part = blockIdx.x / nblk;
    const int64_t cn = (int64_t)a.ch * a.N;
    if (blockIdx.x == 0) seq_check(a.seqs, a.err, tid, kThr);

    BwdBlock<T, NP> k(b);
    k.ckpt = reinterpret_cast<float4 *>(smem);
    k.tile = reinterpret_cast<float4 *>(smem + S::kCkpt);
    float *sB = reinterpret_cast<float *>(smem + S::kCkpt + S::kTile), *sC = sB + kWin * S::kNT;
    int *seq_of = reinterpret_cast<int *>(smem + S::kCkpt + S::kTile + S::kBCBytes), *flag_of = seq_of + kWin;
    k.sB = sB;
    k.sC = sC;
    k.seq_of = seq_of;
    k.flag_of = flag_of;
    k.lane = tid & 31;
    k.warp = tid >> 5;
    k.nl = tid & 3;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        k.dl[r] = (k.warp * R + r) * 8 + (k.lane >> 2);
        k.live[r] = k.dl[r] < ch.n;
        k.dn[r] = (int64_t)(ch.d0 + k.dl[r]) * a.N;
        float t[NP];
        load_states<NP>(t, a.A, k.dn[r], k.nl, a.N, k.live[r]);
#pragma unroll
        for (int i = 0; i < NP; ++i) t[i] *= kLog2e;
        to_pairs<NP>(k.A2[r], t);
#pragma unroll
        for (int i = 0; i < P2; ++i) k.G[r][i] = k.dA[r][i] = 0;
    }
    // empty sequences: their final state is their initial one
    if (b.dh0 != nullptr)
        for (int64_t s = part; s < a.seqs.N; s += a.nchunks)
            if (seq_empty(a.seqs, (int)s))
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float t[NP];
                    load_states<NP>(t, b.dht, s * cn + k.dn[r], k.nl, a.N, k.live[r] && b.dht != nullptr);
                    store_states<NP>(t, b.dh0, s * cn + k.dn[r], k.nl, a.N, k.live[r]);
                }

    const int64_t c0 = part * a.chunk;
    const int64_t c1 = c0 + a.chunk < a.seqs.rows ? c0 + a.chunk : a.seqs.rows;
    const int tr0 = tid >> 3, tc = (tid & 7) * 8;
    const int nc = ch.n - tc;
    const int64_t dc = ch.d0 + tc;
    float accD[8], accb[8];  // over this thread's tokens
#pragma unroll
    for (int j = 0; j < 8; ++j) accD[j] = accb[j] = 0.f;

    f2 hin[R][P2];  // the state before the chunk
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float t[NP];
        load_states<NP>(t, a.hchunk, part * cn + k.dn[r], k.nl, a.N, k.live[r] && part > 0);
        to_pairs<NP>(hin[r], t);
        load_states<NP>(t, b.gchunk, part * cn + k.dn[r], k.nl, a.N, k.live[r] && part + 1 < a.nchunks);
        to_pairs<NP>(k.G[r], t);
    }

    const int64_t windows = c1 > c0 ? (c1 - c0 + kWin - 1) / kWin : 0;
    for (int64_t wi = windows - 1; wi >= 0; --wi) {
        const int64_t w0 = c0 + wi * kWin;
        const int64_t w1 = w0 + kWin < c1 ? w0 + kWin : c1;
        __syncthreads();  // the previous window's results have been read
        for (int tr = tr0; tr < kWin; tr += kRowsAt) {
            const int64_t row = w0 + tr;
            const int n = row < w1 ? nc : 0;
            Raw<T, 8> ru, rdt, rz, rdy;
            load8<T>(ru, a.u, row * a.us + dc, n, a.vec);
            load8<T>(rdt, a.dt, row * a.dts + dc, n, a.vec);
            load8<T>(rdy, b.dy, row * a.ch + dc, n, a.vec);
            if (a.z != nullptr) load8<T>(rz, a.z, row * a.zs + dc, n, a.vec);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = j < n;
                const float bias = a.bias != nullptr && in ? a.bias[dc + j] : 0.f;
                const float delta = in ? step_of<T>(rdt.get(j) + bias, a.softplus) : 0.f;
                float g = in ? rdy.get(j) : 0.f;
                if (a.z != nullptr) g *= in ? act_value(rz.get(j), true) : 0.f;
                k.tile[tr * kDB + slot_of(tc + j)] = make_float4(delta, in ? delta * ru.get(j) : 0.f, g, 0.f);
            }
        }
        for (int e = tid; e < 2 * kWin * S::kNT; e += kThr) {
            const bool isC = e >= kWin * S::kNT;
            const int q = isC ? e - kWin * S::kNT : e;
            const int64_t row = w0 + q / S::kNT;
            const int n = q % S::kNT;
            float v = 0.f;
            if (row < w1 && n < a.N)
                v = to_f(static_cast<const T *>(isC ? a.C : a.B)[row * (isC ? a.cs : a.bs) + (int64_t)ch.g * a.N + n]);
            sB[e] = v;  // sC follows sB
        }
        const SeqAt last = seq_find(a.seqs, w1 - 1);
        const bool ragged = !(last.start < w0 && last.end > w1);  // a sequence starts or ends here
        if (ragged && tid < kWin) {
            const int64_t row = w0 + tid;
            int s = 0, f = 0;
            if (row < w1) {
                const SeqAt at = seq_find(a.seqs, row);
                s = at.s;
                f = (row == at.start ? 1 : 0) | (row + 1 == at.end ? 2 : 0);
            }
            seq_of[tid] = s;
            flag_of[tid] = f;
        }
        // the state before the window
        f2 h[R][P2];
        const bool fix = wi > 0 && seq_find(a.seqs, w0 - 1).start < c0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (wi == 0) {
#pragma unroll
                for (int i = 0; i < P2; ++i) h[r][i] = hin[r][i];
            } else {
                float t[NP];
                load_states<NP>(t, b.hwin, (w0 / kWin) * cn + k.dn[r], k.nl, a.N, k.live[r]);
                to_pairs<NP>(h[r], t);
                if (fix) {
                    const float sw = k.live[r] ? b.swin[(w0 / kWin) * a.ch + ch.d0 + k.dl[r]] : 0.f;
                    const f2 s2 = pk(sw, sw);
#pragma unroll
                    for (int i = 0; i < P2; ++i) h[r][i] = fma2(exp2_2(mul2(s2, k.A2[r][i])), hin[r][i], h[r][i]);
                }
            }
        }
        __syncthreads();
        if (ragged) {
            k.template forward<true>(h);
            for (int g = kGroups - 1; g >= 0; --g) k.template backward<true>(g);
        } else {
            k.template forward<false>(h);
            for (int g = kGroups - 1; g >= 0; --g) k.template backward<false>(g);
        }
        __syncthreads();
        // dB, dC of this block's channels: the warps' sums in order
        for (int e = tid; e < kWin * 2 * S::kNT; e += kThr) {
            const int t = e / (2 * S::kNT), q = e % (2 * S::kNT), n = q % S::kNT;
            if (w0 + t < w1 && n < a.N) {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < S::kWarps; ++w)
                    v += reinterpret_cast<const float *>(k.ckpt + ((t / 4) * S::kWarps + w) * (S::E / 4) * 32)[(t % 4) * 2 * S::kNT + q];
                const int64_t row = ((int64_t)(blk % a.blocks_per_group) * a.seqs.rows + w0 + t) * a.G + ch.g;
                b.pbc[(row * 2 + q / S::kNT) * a.N + n] = v;
            }
        }
        // per (token, channel)
        for (int tr = tr0; tr < kWin; tr += kRowsAt) {
            const int64_t row = w0 + tr;
            if (row >= w1 || nc <= 0) continue;
            Raw<T, 8> ru, rdt, rz, rdy;
            load8<T>(ru, a.u, row * a.us + dc, nc, a.vec);
            load8<T>(rdt, a.dt, row * a.dts + dc, nc, a.vec);
            load8<T>(rdy, b.dy, row * a.ch + dc, nc, a.vec);
            if (a.z != nullptr) load8<T>(rz, a.z, row * a.zs + dc, nc, a.vec);
            float du[8], ddt[8], dz[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = j < nc;
                const float4 q = k.tile[tr * kDB + slot_of(tc + j)];  // s, w, y
                const float raw = rdt.get(j) + (a.bias != nullptr && in ? a.bias[dc + j] : 0.f);
                const float delta = step_of<T>(raw, a.softplus), u = ru.get(j);
                const float D = a.D != nullptr && in ? a.D[dc + j] : 0.f;
                float val = 1.f, der = 0.f;
                if (a.z != nullptr) act_both(rz.get(j), true, val, der);
                const float g = rdy.get(j) * val;
                du[j] = fmaf(D, g, delta * q.x);
                ddt[j] = fmaf(u, q.x, q.y);
                if (a.softplus) ddt[j] *= sigmoid(raw);
                dz[j] = rdy.get(j) * fmaf(D, u, q.z) * der;
                accD[j] = fmaf(g, u, accD[j]);
                accb[j] += ddt[j];
            }
            store8<T>(b.du, row * a.ch + dc, du, nc, a.vec);
            store8<T>(b.ddt, row * a.ch + dc, ddt, nc, a.vec);
            if (b.dz != nullptr) store8<T>(b.dz, row * a.ch + dc, dz, nc, a.vec);
        }
    }
    // sums over this chunk's tokens
    float *part_out = b.partial + part * (cn + 2 * (int64_t)a.ch);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float t[NP];
        from_pairs<NP>(t, k.dA[r]);
        store_states<NP>(t, part_out, k.dn[r], k.nl, a.N, k.live[r]);
    }
    __syncthreads();
    float *red = reinterpret_cast<float *>(smem);  // [kRowsAt][2][kDB]
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        red[(tr0 * 2 + 0) * kDB + tc + j] = accD[j];
        red[(tr0 * 2 + 1) * kDB + tc + j] = accb[j];
    }
    __syncthreads();
    for (int e = tid; e < 2 * kDB; e += kThr) {
        const int which = e / kDB, c = e % kDB;
        if (c < ch.n) {
            float v = 0.f;
            for (int i = 0; i < kRowsAt; ++i) v += red[(i * 2 + which) * kDB + c];
            part_out[cn + (int64_t)which * a.ch + ch.d0 + c] = v;
        }
    }
}

// dB and dC from the blocks' shares, in order: one thread per (row, group, state) and tensor.
template <typename T>
__global__ void __launch_bounds__(256) scan_bwd_bc_kernel(const BwdArgs b) {
    const ScanArgs &a = b.f;
    const int64_t per = a.seqs.rows * a.G * 2 * a.N;
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= per) return;
    float s = 0.f;
#pragma unroll 4
    for (int k = 0; k < a.blocks_per_group; ++k) s += b.pbc[k * per + e];
    const int64_t row = e / (2 * a.N);  // row * G + group
    const int q = (int)(e % (2 * a.N));
    static_cast<T *>(q < a.N ? b.dB : b.dC)[row * a.N + (q < a.N ? q : q - a.N)] = from_f<T>(s);
}

template <typename T, int NP>
cudaError_t launch_np(const BwdArgs &b, cudaStream_t stream) {
    const ScanArgs &a = b.f;
    const int64_t nblk = (int64_t)a.G * a.blocks_per_group;
    if (nblk * a.nchunks > INT32_MAX) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)(nblk * a.nchunks);
    cudaError_t e = cudaFuncSetAttribute(scan_bwd_kernel<T, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, BwdShape<NP>::kSmem);
    if (e != cudaSuccess) return e;
    if (a.seqs.rows > kWin) {  // one window: nothing to hand over
        if constexpr (NP == 2)
            e = launch_local<T, 8, 1>(b, stream);
        else
            e = launch_local<T, 16, NP / 4>(b, stream);
        if (e != cudaSuccess) return e;
    }
    if (a.nchunks > 1) {
        e = launch_scan_carry(a, stream);
        if (e != cudaSuccess) return e;
        scan_bwd_carry_kernel<<<(unsigned)ceil_div((int64_t)a.ch * a.N, 256), 256, 0, stream>>>(b);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    scan_bwd_kernel<T, NP><<<grid, BwdShape<NP>::kThr, BwdShape<NP>::kSmem, stream>>>(b);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t per = a.seqs.rows * a.G * 2 * a.N;
    if (per > 0) scan_bwd_bc_kernel<T><<<(unsigned)ceil_div(per, 256), 256, 0, stream>>>(b);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bwd_t(const BwdArgs &b, cudaStream_t stream) {
    switch (np_of(b.f.N)) {
        case 2:
            return launch_np<T, 2>(b, stream);
        case 4:
            return launch_np<T, 4>(b, stream);
        case 8:
            return launch_np<T, 8>(b, stream);
        default:
            return launch_np<T, 16>(b, stream);
    }
}

int elem_size(int dtype) { return dtype == KDA_DTYPE_BF16 ? 2 : 4; }

int bwd_check(const kda_scan_bwd_params &p) {
    const int st = scan_check(p.f);
    if (st != KDA_OK) return st;
    if (p.dA == nullptr || (p.f.T != 0 && (p.dy == nullptr || p.du == nullptr || p.ddt == nullptr || p.dB == nullptr || p.dC == nullptr)))
        return KDA_ERR_INVALID_ARG;
    if ((p.dD != nullptr && p.f.D == nullptr) || (p.dz != nullptr && p.f.z == nullptr)) return KDA_ERR_INVALID_ARG;
    const size_t e = elem_size(p.f.dtype);
    const void *data[] = {p.dy, p.du, p.ddt, p.dB, p.dC, p.dz};
    for (const void *q : data)
        if (!aligned(q, e)) return KDA_ERR_ALIGNMENT;
    const void *f32[] = {p.dht, p.dA, p.dD, p.ddt_bias, p.dh0};
    for (const void *q : f32)
        if (!aligned(q, 4)) return KDA_ERR_ALIGNMENT;
    return KDA_OK;
}

// Chunks: about four blocks of the third step per SM slot, of whole windows.
struct BwdPlan {
    int64_t chunk, nchunks, windows, rows, bpg;
    size_t h, g, s, hw, sw, pbc, partial, bytes;  // offsets in floats, then the size in bytes
};
BwdPlan bwd_plan(const kda_scan_params &p) {
    BwdPlan q{};
    q.rows = p.cu_seqlens != nullptr ? (int64_t)p.T : (int64_t)p.batch * p.T;
    q.bpg = ceil_div(p.channels / p.G, kDB);
    const int64_t nblk = p.G * q.bpg;
    const int64_t sms = sm_count() > 0 ? sm_count() : 1;
    int64_t n = ceil_div(12 * sms, nblk);
    q.chunk = ceil_div(ceil_div(q.rows > 0 ? q.rows : 1, n), kWin) * kWin;
    q.nchunks = ceil_div(q.rows, q.chunk);
    if (q.nchunks < 1) q.nchunks = 1;
    q.windows = ceil_div(q.rows, kWin);
    const size_t cn = (size_t)p.channels * p.N, ch = p.channels;
    size_t at = 0;
    auto take = [&](size_t n2) {
        const size_t here = at;
        at += (n2 + 3) / 4 * 4;
        return here;
    };
    q.h = take(q.nchunks * cn);
    q.g = take(q.nchunks * cn);
    q.s = take(q.nchunks * ch);
    q.hw = take(q.windows * cn);
    q.sw = take(q.windows * ch);
    q.pbc = take((size_t)q.bpg * q.rows * p.G * 2 * p.N);
    q.partial = take(q.nchunks * (cn + 2 * ch));
    q.bytes = at * sizeof(float);
    return q;
}

}  // namespace
}  // namespace scan
}  // namespace kda

extern "C" {

size_t kda_scan_bwd_workspace(const kda_scan_bwd_params *p) {
    using namespace kda::scan;
    return p == nullptr || bwd_check(*p) != KDA_OK ? 0 : bwd_plan(p->f).bytes;
}

int kda_scan_bwd(const kda_scan_bwd_params *p, cudaStream_t stream) {
    using namespace kda;
    using namespace kda::scan;
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    const int st = bwd_check(*p);
    if (st != KDA_OK) return st;
    const BwdPlan q = bwd_plan(p->f);
    if (p->workspace != nullptr && p->workspace_bytes < q.bytes) return KDA_ERR_INVALID_ARG;
    if (!aligned(p->workspace, 16)) return KDA_ERR_ALIGNMENT;
    const void *more[] = {p->dy, p->du, p->ddt, p->dz};
    BwdArgs b{};
    b.f = scan_args(p->f, more, 4);
    b.f.chunk = q.chunk;
    b.f.nchunks = q.nchunks;
    b.f.vec_states = aligned(p->f.A, 16) && aligned(p->f.h0, 16) && aligned(p->dht, 16) && p->f.N % 4 == 0;
    b.dy = p->dy;
    b.dht = p->dht;
    b.du = p->du;
    b.ddt = p->ddt;
    b.dB = p->dB;
    b.dC = p->dC;
    b.dz = p->dz;
    b.dh0 = p->dh0;
    cudaError_t e = device_error_word(&b.f.err);
    if (e != cudaSuccess) return status_of_cuda(e);
    Scratch ws;
    e = ws.get(p->workspace, q.bytes, stream);
    if (e != cudaSuccess) return status_of_cuda(e);
    float *base = static_cast<float *>(ws.ptr);
    b.f.hchunk = base + q.h;
    b.gchunk = base + q.g;
    b.f.schunk = base + q.s;
    b.hwin = base + q.hw;
    b.swin = base + q.sw;
    b.pbc = base + q.pbc;
    b.partial = base + q.partial;
    e = p->f.dtype == KDA_DTYPE_BF16 ? launch_bwd_t<bf16>(b, stream) : launch_bwd_t<float>(b, stream);
    if (e == cudaSuccess) {
        const int64_t cn = (int64_t)p->f.channels * p->f.N;
        const SumOuts outs{{p->dA, p->dD, p->ddt_bias, nullptr}, {cn, p->f.channels, p->f.channels, 0}};
        e = launch_sum_partials(b.partial, q.nchunks, cn + 2 * (int64_t)p->f.channels, outs, stream);
    }
    return status_of_cuda(ws.release(e));
}

}  // extern "C"
