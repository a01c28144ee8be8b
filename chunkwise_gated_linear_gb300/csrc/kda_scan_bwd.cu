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
//      It leaves the local state at every 16 rows (a window; 8 above 32 states), the chunk's end state, its adjoint
//      at the start from a zero adjoint at the end (in the same forward walk:
//      sum_t (a_c0 .. a_t) C_t g_t), and sums of delta.
//   2. scan_bwd_carry_kernel: true states at the chunk starts, true adjoints at the ends.
//   3. scan_bwd_kernel: per chunk and 64 channels, windows last to first. A window's start state
//      is its local state plus exp(A sum delta) times the chunk's start state; from there the
//      states before every group of two tokens go to shared memory, and the groups are taken
//      last to first: a and a h_{t-1} of their tokens in registers, then backwards.
// Sums over the states go across 4 lanes, sums over channels across 8 lanes (one exchange per
// value and halving, so that each lane ends with one total), then over warps and blocks in a
// fixed order. Bound by issue: about 11 instructions per (token, channel, state) in the first kernel, 37 in the
// third. 2 x 4096 tokens of 4096 channels, 16 states, bf16: 1075 us, of which 236 and 780.
#include <type_traits>

#include "scan_common.cuh"

namespace kda {
namespace scan {

namespace {

// Tokens per window: what the third kernel keeps states of in shared memory. With 16 states, windows of 16
// and groups of two tokens leave registers and shared memory for four blocks per SM (2 x 4096 tokens
// of 4096 channels: 1072 us); windows of 32 and groups of four for three (1120 us).
__host__ __device__ constexpr int win_of(int np) { return np <= 8 ? 16 : 8; }
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
template <typename T, int NS, int LN, int WIN>
__global__ void __launch_bounds__(kLThr, 4) scan_bwd_local_kernel(const BwdArgs b) {
    constexpr int kNT = NS * LN, P2 = NS / 2, kChan = kLThr / LN;
    constexpr int kTile = 32;  // tokens of B and C in shared memory
    constexpr int kBC = 2 * kTile * kNT / kLThr;
    __shared__ __align__(16) float sB[kTile * kNT], sC[kTile * kNT];
    const ScanArgs &a = b.f;
    const int tid = threadIdx.x;
    const int nblk = a.G * a.blocks_per_group;
    const int blk = blockIdx.x % nblk;
    const int64_t part = blockIdx.x / nblk;
    const int g = blk / a.blocks_per_group;
    const int first = (blk % a.blocks_per_group) * kChan + tid / LN;
    const int n0 = (tid % LN) * NS;
    const bool live = first < a.chg;
    const uint32_t d = g * a.chg + (live ? first : 0);
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
    // The chunk's start adjoint is that of the sequence which holds its first row: it is complete, and leaves,
    // where that sequence or the chunk ends, with dht (if the sequence ends) through the decays since
    // the chunk's start. What f and P become in later sequences of the chunk is not used. (Were
    // they held at zero instead, an infinity there would come back as NaN in the sequence before.)
    auto open = [&] { return at.start <= c0; };
    auto leave = [&](bool ends) {
        if (ends && b.dht != nullptr) {
            f2 t[P2];
            get_states<NS>(t, b.dht, at.s * cn + dn, n0, a.N, live, vst);
#pragma unroll
            for (int i = 0; i < P2; ++i) f[i] = fma2(P[i], t[i], f[i]);
        }
        put_states<NS>(f, b.gchunk, part * cn + dn, n0, a.N, live, a.N == kNT);
    };
    const float bias = a.bias != nullptr ? a.bias[d] : 0.f;
    const bool gate = a.z != nullptr;

    T nu[4], ndt[4], ndy[4], nz[4];
    auto fetch = [&](int64_t r0) {
        // the rows' places are the same for all threads
        const T *pu = static_cast<const T *>(a.u) + r0 * a.us, *pd = static_cast<const T *>(a.dt) + r0 * a.dts;
        const T *py = static_cast<const T *>(b.dy) + r0 * a.ch, *pz = static_cast<const T *>(a.z) + r0 * a.zs;
        if (r0 + 4 <= c1) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                nu[k] = (pu + k * a.us)[d];
                ndt[k] = (pd + k * a.dts)[d];
                ndy[k] = (py + (int64_t)k * a.ch)[d];
                if (gate) nz[k] = (pz + k * a.zs)[d];
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (r0 + k < c1) {
                    nu[k] = (pu + k * a.us)[d];
                    ndt[k] = (pd + k * a.dts)[d];
                    ndy[k] = (py + (int64_t)k * a.ch)[d];
                    if (gate) nz[k] = (pz + k * a.zs)[d];
                }
        }
    };
    float nbc[kBC];
    auto fetch_bc = [&](int64_t t0) {
#pragma unroll
        for (int k = 0; k < kBC; ++k) {
            const bool isC = k >= kBC / 2;
            const int e = (tid + k * kLThr) % (kTile * kNT);
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
            const f2 e0 = decay2(d2, A2[i]), e1 = decay2(d2, A2[i + 1]);
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
    for (int64_t t0 = c0; t0 < c1; t0 += kTile) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kBC; ++k) (k < kBC / 2 ? sB : sC)[(tid + k * kLThr) % (kTile * kNT)] = nbc[k];
        __syncthreads();
        if (t0 + kTile < c1) fetch_bc(t0 + kTile);
#pragma unroll 1
        for (int t = 0; t < kTile; t += 4) {
            const int64_t r = t0 + t;
            if (r >= c1) break;
            if (t % WIN == 0 && r > c0) {  // the state before a window
                put_states<NS>(h, b.hwin, (r / WIN) * cn + dn, n0, a.N, live, a.N == kNT);
                if (live && n0 == 0) b.swin[(r / WIN) * a.ch + d] = S;
            }
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
                        if (open()) leave(true);
                        seq_next(a.seqs, at);
                        get_states<NS>(h, a.h0, at.s * cn + dn, n0, a.N, live && a.h0 != nullptr, vst);
                    }
                    token(t + k, cu_[k], cdt[k], cdy[k], cz[k]);
                }
            }
        }
    }
    if (open()) leave(c1 == at.end);
    put_states<NS>(h, a.hchunk, part * cn + dn, n0, a.N, live, a.N == kNT);
    if (live && n0 == 0) a.schunk[part * a.ch + d] = S;
}

template <typename T, int NS, int LN, int WIN>
cudaError_t launch_local(BwdArgs b, cudaStream_t stream) {
    b.f.blocks_per_group = (int)ceil_div(b.f.chg, kLThr / LN);
    const int64_t grid = b.f.nchunks * b.f.G * b.f.blocks_per_group;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    scan_bwd_local_kernel<T, NS, LN, WIN><<<(unsigned)grid, kLThr, 0, stream>>>(b);
    return cudaGetLastError();
}

// ---- 2: between the chunks, in place ----------------------------------------------------------
// Adjoints: the adjoint that enters chunk c - 1 at its end is chunk
// c's local one plus, when no sequence ends in chunk c, exp(A sum delta) times what enters c.
__device__ __forceinline__ void carry_adjoints(const BwdArgs &b) {
    const ScanArgs &a = b.f;
    constexpr int kAhead = 16;
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

// Both ways at once: half the blocks each.
__global__ void __launch_bounds__(256) scan_bwd_carry_kernel(const BwdArgs b) {
    if (blockIdx.y == 0)
        carry_states(b.f);
    else
        carry_adjoints(b);
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

// A block: 128 threads, 64 channels. Warp w has channels 16 w .. 16 w + 15: thread (dl, nl) = (lane / 4,
// lane % 4) has channels 16 w + dl and 16 w + 8 + dl, as the two halves of every pair, and states
// nl NP .. nl NP + NP - 1 of both: step sizes, inputs and gradients of a pair come as pairs, B and C (the
// same for all channels) are doubled in registers (doubled in shared memory they took a quarter of
// the load/store wavefronts: 1104 us for the sizes above where this then took 1080).
template <int NP>
struct BwdShape {
    static constexpr int kThr = 128, kWarps = 4;
    static constexpr int kNT = kLN * NP;
    static constexpr int kWin = win_of(NP);
    // tokens whose decays are held in registers while they are walked back
    static constexpr int kSC = NP <= 8 ? 2 : 1;
    static constexpr int kGroups = kWin / kSC;
    static constexpr int kCkpt = kGroups * 2 * NP * kThr * 4;  // states before every group of tokens
    static constexpr int kTileA = kWin * 32 * 16;              // delta and x of a pair; then s and w
    static constexpr int kTileG = kWin * 32 * 8;               // g; then y
    static constexpr int kTileD = kWin * 32 * 8;               // delta
    static constexpr int kBCBytes = 2 * kWin * kNT * 4;
    static constexpr int kFlags = kWin * 8;                    // per row: sequence, start / end bits
    static constexpr int kPar = 2 * kDB * 4;                   // dt_bias and D of the channels
    static constexpr int kSmem = kCkpt + kTileA + kTileG + kTileD + kBCBytes + kFlags + kPar;
};

// Place of pair dl of warp w in a tile's row t: rotated so that the threads that fill a tile row by row
// (8 channels of one half each) do not all meet in the same banks.
__device__ __forceinline__ int pair_slot(int t, int w, int dl) { return w * 8 + ((dl ^ (w + 4 * (t & 1))) & 7); }

template <typename T, int NP>
struct BwdBlock {
    using S = BwdShape<NP>;
    const BwdArgs &b;
    float4 *tileA;       // [kWin][32]
    float2 *tileG;       // [kWin][32]
    const float *sB, *sC;   // [kWin][kNT]
    float4 *ckpt;        // [kGroups][kWarps][NP / 2][32]
    const int *seq_of, *flag_of;
    int lane, warp, nl, dl;
    int64_t dn0, dn1;    // the two channels' places in [ch][N]
    bool live0, live1;
    f2 A2[NP], G[NP], dA[NP];

    __device__ __forceinline__ BwdBlock(const BwdArgs &args) : b(args) {}
    __device__ __forceinline__ float4 *group_mem(int g) const { return ckpt + (g * S::kWarps + warp) * (NP / 2) * 32; }
    // the pair's states at `at` (of [..][ch][N])
    __device__ __forceinline__ void states(f2 (&h)[NP], const float *base, int64_t at) const {
        float lo[NP], hi[NP];
        load_states<NP>(lo, base, at + dn0, nl, b.f.N, live0 && base != nullptr);
        load_states<NP>(hi, base, at + dn1, nl, b.f.N, live1 && base != nullptr);
#pragma unroll
        for (int i = 0; i < NP; ++i) h[i] = pk(lo[i], hi[i]);
    }
    __device__ __forceinline__ void put(const f2 (&h)[NP], float *base, int64_t at) const {
        float lo[NP], hi[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) upk(h[i], lo[i], hi[i]);
        store_states<NP>(lo, base, at + dn0, nl, b.f.N, live0);
        store_states<NP>(hi, base, at + dn1, nl, b.f.N, live1);
    }
    __device__ __forceinline__ int64_t seq_at(int t) const { return seq_of[t] * (int64_t)b.f.ch * b.f.N; }
    __device__ __forceinline__ void row_bc(f2 (&v)[NP], const float *s, int t) const {
        float f[NP];
        if constexpr (NP >= 4) {
#pragma unroll
            for (int i = 0; i < NP / 4; ++i) {
                const float4 q = reinterpret_cast<const float4 *>(s + t * S::kNT + nl * NP)[i];
                f[4 * i] = q.x;
                f[4 * i + 1] = q.y;
                f[4 * i + 2] = q.z;
                f[4 * i + 3] = q.w;
            }
        } else {
            const float2 q = *reinterpret_cast<const float2 *>(s + t * S::kNT + nl * NP);
            f[0] = q.x;
            f[1] = q.y;
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) v[i] = pk(f[i], f[i]);
    }
    // delta and x of the pair at token t
    __device__ __forceinline__ void row_dx(f2 &d2, f2 &x2, int t) const {
        const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(&tileA[t * 32 + pair_slot(t, warp, dl)]);
        d2 = q.x;
        x2 = q.y;
    }
    // states before every group of tokens into shared memory, from the state h before the window
    template <bool RAG>
    __device__ __forceinline__ void forward(f2 (&h)[NP]) const {
#pragma unroll 1
        for (int g = 0; g < S::kGroups; ++g) {
            float4 *to = group_mem(g);
#pragma unroll
            for (int q = 0; q < NP / 2; ++q) *reinterpret_cast<ulonglong2 *>(&to[q * 32 + lane]) = make_ulonglong2(h[2 * q], h[2 * q + 1]);
            if (g == S::kGroups - 1) break;
#pragma unroll
            for (int k = 0; k < S::kSC; ++k) {
                const int t = S::kSC * g + k;
                if (RAG && (flag_of[t] & 1)) states(h, b.f.h0, seq_at(t));
                f2 B[NP], d2, x2;
                row_bc(B, sB, t);
                row_dx(d2, x2, t);
#pragma unroll
                for (int i = 0; i < NP; ++i) h[i] = fma2(decay2(d2, A2[i]), h[i], mul2(x2, B[i]));
            }
        }
    }
    // the tokens of group g, last to first
    template <bool RAG>
    __device__ __forceinline__ void backward(int g) {
        float4 *mem = group_mem(g);
        f2 h[NP], e[S::kSC][NP], eh[S::kSC][NP];
#pragma unroll
        for (int q = 0; q < NP / 2; ++q) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(&mem[q * 32 + lane]);
            h[2 * q] = v.x;
            h[2 * q + 1] = v.y;
        }
#pragma unroll
        for (int k = 0; k < S::kSC; ++k) {
            const int t = S::kSC * g + k;
            if (RAG && (flag_of[t] & 1)) states(h, b.f.h0, seq_at(t));
            f2 B[NP], d2, x2;
            row_bc(B, sB, t);
            row_dx(d2, x2, t);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                e[k][i] = decay2(d2, A2[i]);
                eh[k][i] = mul2(e[k][i], h[i]);
                h[i] = fma2(x2, B[i], eh[k][i]);
            }
        }
        __syncwarp();  // the group's states have been read: its memory takes dB and dC
#pragma unroll
        for (int k = S::kSC - 1; k >= 0; --k) {
            const int t = S::kSC * g + k;
            if (RAG && (flag_of[t] & 2)) states(G, b.dht, seq_at(t));
            f2 B[NP], C[NP], d2, x2, s2 = 0, w2 = 0, y2 = 0;
            row_bc(B, sB, t);
            row_bc(C, sC, t);
            row_dx(d2, x2, t);
            const int at = t * 32 + pair_slot(t, warp, dl);
            const f2 g2 = *reinterpret_cast<const f2 *>(&tileG[at]);
            float vb[NP], vc[NP];  // the pair's share of dB and dC
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const f2 l = fma2(g2, C[i], G[i]);
                const f2 ht = fma2(x2, B[i], eh[k][i]);
                const f2 q = mul2(l, eh[k][i]);
                vb[i] = hsum2(mul2(l, x2));
                vc[i] = hsum2(mul2(ht, g2));
                s2 = i == 0 ? mul2(l, B[i]) : fma2(l, B[i], s2);
                y2 = i == 0 ? mul2(ht, C[i]) : fma2(ht, C[i], y2);
                w2 = i == 0 ? mul2(q, A2[i]) : fma2(q, A2[i], w2);
                dA[i] = fma2(q, d2, dA[i]);
                G[i] = mul2(l, e[k][i]);
            }
            if (RAG && (flag_of[t] & 1) && b.dh0 != nullptr) put(G, b.dh0, seq_at(t));
            // over the states: lane nl gets s of the first, of the second channel, w of the first, of the second
            float v4[4], y0, y1;
            upk(s2, v4[0], v4[1]);
            upk(w2, v4[2], v4[3]);
            upk(y2, y0, y1);
            const float sw = sum_lanes(v4, nl);
            const bool odd = nl & 1;
            float yy = (odd ? y1 : y0) + __shfl_xor_sync(0xffffffffu, odd ? y0 : y1, 1);
            yy += __shfl_xor_sync(0xffffffffu, yy, 2);
            __syncwarp();  // all four lanes have read this token's tile words
            reinterpret_cast<float *>(&tileA[at])[nl] = nl < 2 ? sw : sw * kLn2;
            if (nl < 2) reinterpret_cast<float *>(&tileG[at])[nl] = yy;
            // over this warp's channels: [which][4 NP] of token t
            float *to = reinterpret_cast<float *>(mem) + k * 2 * S::kNT;
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
    }
};

template <typename T, int NP>
__global__ void __launch_bounds__(BwdShape<NP>::kThr, NP <= 4 ? 4 : 1) scan_bwd_kernel(const BwdArgs b) {
    using S = BwdShape<NP>;
    constexpr int kThr = S::kThr, kWin = S::kWin;
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
    unsigned char *mem = smem;
    auto take = [&](int bytes) {
        unsigned char *p = mem;
        mem += bytes;
        return p;
    };
    k.ckpt = reinterpret_cast<float4 *>(take(S::kCkpt));
    k.tileA = reinterpret_cast<float4 *>(take(S::kTileA));
    k.tileG = reinterpret_cast<float2 *>(take(S::kTileG));
    float *tileD = reinterpret_cast<float *>(take(S::kTileD));
    float *sB = reinterpret_cast<float *>(take(S::kBCBytes));
    int *seq_of = reinterpret_cast<int *>(take(S::kFlags)), *flag_of = seq_of + kWin;
    float *sbias = reinterpret_cast<float *>(take(S::kPar)), *sD = sbias + kDB;
    if (tid < kDB) {
        sbias[tid] = a.bias != nullptr && tid < ch.n ? a.bias[ch.d0 + tid] : 0.f;
        sD[tid] = a.D != nullptr && tid < ch.n ? a.D[ch.d0 + tid] : 0.f;
    }
    k.sB = sB;
    k.sC = k.sB + kWin * S::kNT;
    k.seq_of = seq_of;
    k.flag_of = flag_of;
    k.lane = tid & 31;
    k.warp = tid >> 5;
    k.nl = tid & 3;
    k.dl = k.lane >> 2;
    const int own = k.warp * 16 + k.dl;  // and own + 8
    k.live0 = own < ch.n;
    k.live1 = own + 8 < ch.n;
    k.dn0 = (int64_t)(ch.d0 + own) * a.N;
    k.dn1 = k.dn0 + 8 * (int64_t)a.N;
    k.states(k.A2, a.A, 0);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        k.A2[i] = mul2(k.A2[i], pk(kLog2e, kLog2e));
        k.dA[i] = 0;
    }
    // empty sequences: their final state is their initial one
    if (b.dh0 != nullptr)
        for (int64_t s = part; s < a.seqs.N; s += a.nchunks)
            if (seq_empty(a.seqs, (int)s)) {
                f2 t[NP];
                k.states(t, b.dht, s * cn);
                k.put(t, b.dh0, s * cn);
            }

    const int64_t c0 = part * a.chunk;
    const int64_t c1 = c0 + a.chunk < a.seqs.rows ? c0 + a.chunk : a.seqs.rows;
    const int tr0 = tid >> 3, tc = (tid & 7) * 8;
    const int tw = tc >> 4, half = (tc >> 3) & 1;  // whose pairs these 8 channels belong to, and which half
    const int nc = ch.n - tc;
    const int64_t dc = ch.d0 + tc;
    float accD[8], accb[8];  // over this thread's tokens
#pragma unroll
    for (int j = 0; j < 8; ++j) accD[j] = accb[j] = 0.f;
    k.states(k.G, part + 1 < a.nchunks ? b.gchunk : nullptr, part * cn);

    const int64_t windows = c1 > c0 ? (c1 - c0 + kWin - 1) / kWin : 0;
    for (int64_t wi = windows - 1; wi >= 0; --wi) {
        const int64_t w0 = c0 + wi * kWin;
        const int64_t w1 = w0 + kWin < c1 ? w0 + kWin : c1;
        __syncthreads();  // the previous window's results have been read
        // ALL: the row and its eight channels exist
        auto stage = [&](auto all, int tr, int64_t row, int n) {
            constexpr bool ALL = decltype(all)::value;
            Raw<T, 8> ru, rdt, rz, rdy;
            load8<T>(ru, a.u, row * a.us + dc, n, a.vec);
            load8<T>(rdt, a.dt, row * a.dts + dc, n, a.vec);
            load8<T>(rdy, b.dy, row * a.ch + dc, n, a.vec);
            if (a.z != nullptr) load8<T>(rz, a.z, row * a.zs + dc, n, a.vec);
            float bias[8];
            load_vec<float, 8>(bias, sbias + tc);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = ALL || j < n;
                const float delta = in ? step_of<T>(rdt.get(j) + bias[j], a.softplus) : 0.f;
                float g = in ? rdy.get(j) : 0.f;
                if (a.z != nullptr) g *= in ? act_value(rz.get(j), true) : 0.f;
                const int at = tr * 32 + pair_slot(tr, tw, j);
                reinterpret_cast<float *>(&k.tileA[at])[half] = delta;
                reinterpret_cast<float *>(&k.tileA[at])[2 + half] = in ? delta * ru.get(j) : 0.f;
                reinterpret_cast<float *>(&k.tileG[at])[half] = g;
                tileD[2 * at + half] = delta;
            }
        };
        for (int tr = tr0; tr < kWin; tr += kRowsAt) {
            const int64_t row = w0 + tr;
            if (row < w1 && nc >= 8)
                stage(std::true_type{}, tr, row, 8);
            else
                stage(std::false_type{}, tr, row, row < w1 ? nc : 0);
        }
        for (int e = tid; e < 2 * kWin * S::kNT; e += kThr) {
            const bool isC = e >= kWin * S::kNT;
            const int q = isC ? e - kWin * S::kNT : e;
            const int64_t row = w0 + q / S::kNT;
            const int n = q % S::kNT;
            float v = 0.f;
            if (row < w1 && n < a.N)
                v = to_f(static_cast<const T *>(isC ? a.C : a.B)[row * (isC ? a.cs : a.bs) + (int64_t)ch.g * a.N + n]);
            sB[e] = v;  // C follows B
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
        // the state before the window: local, plus what the chunk's start state leaves of itself
        f2 h[NP];
        if (wi == 0) {
            k.states(h, part > 0 ? a.hchunk : nullptr, part * cn);
        } else {
            const int64_t win = w0 / kWin;
            k.states(h, b.hwin, win * cn);
            if (part > 0 && seq_find(a.seqs, w0 - 1).start < c0) {
                f2 in[NP];
                k.states(in, a.hchunk, part * cn);
                const float *sw = b.swin + win * a.ch + ch.d0 + own;
                const f2 s2 = pk(k.live0 ? sw[0] : 0.f, k.live1 ? sw[8] : 0.f);
#pragma unroll
                for (int i = 0; i < NP; ++i) h[i] = fma2(exp2_2(mul2(s2, k.A2[i])), in[i], h[i]);
            }
        }
        __syncthreads();
        if (ragged) {
            k.template forward<true>(h);
#pragma unroll 1
            for (int g = S::kGroups - 1; g >= 0; --g) k.template backward<true>(g);
        } else {
            k.template forward<false>(h);
#pragma unroll 1
            for (int g = S::kGroups - 1; g >= 0; --g) k.template backward<false>(g);
        }
        __syncthreads();
        // dB, dC of this block's channels: the warps' sums in order
        for (int e = tid; e < kWin * 2 * S::kNT; e += kThr) {
            const int t = e / (2 * S::kNT), q = e % (2 * S::kNT), n = q % S::kNT;
            if (w0 + t < w1 && n < a.N) {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < S::kWarps; ++w)
                    v += reinterpret_cast<const float *>(k.ckpt + ((t / S::kSC) * S::kWarps + w) * (NP / 2) * 32)[(t % S::kSC) * 2 * S::kNT + q];
                const int64_t row = ((int64_t)(blk % a.blocks_per_group) * a.seqs.rows + w0 + t) * a.G + ch.g;
                b.pbc[(row * 2 + q / S::kNT) * a.N + n] = v;
            }
        }
        // per (token, channel); channels that do not exist are computed and not stored
        for (int tr = tr0; tr < kWin; tr += kRowsAt) {
            const int64_t row = w0 + tr;
            if (row >= w1 || nc <= 0) continue;
            Raw<T, 8> ru, rdt, rz, rdy;
            load8<T>(ru, a.u, row * a.us + dc, nc, a.vec);
            load8<T>(rdt, a.dt, row * a.dts + dc, nc, a.vec);
            load8<T>(rdy, b.dy, row * a.ch + dc, nc, a.vec);
            if (a.z != nullptr) load8<T>(rz, a.z, row * a.zs + dc, nc, a.vec);
            float du[8], ddt[8], dz[8], bias[8], D[8];
            load_vec<float, 8>(bias, sbias + tc);
            load_vec<float, 8>(D, sD + tc);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int at = tr * 32 + pair_slot(tr, tw, j);
                const float s = reinterpret_cast<const float *>(&k.tileA[at])[half];
                const float w = reinterpret_cast<const float *>(&k.tileA[at])[2 + half];
                const float y = reinterpret_cast<const float *>(&k.tileG[at])[half];
                const float delta = tileD[2 * at + half], u = ru.get(j);
                float val = 1.f, der = 0.f;
                if (a.z != nullptr) act_both(rz.get(j), true, val, der);
                const float g = rdy.get(j) * val;
                du[j] = fmaf(D[j], g, delta * s);
                ddt[j] = fmaf(u, s, w);
                if (a.softplus) ddt[j] *= sigmoid(rdt.get(j) + bias[j]);
                dz[j] = rdy.get(j) * fmaf(D[j], u, y) * der;
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
    k.put(k.dA, part_out, 0);
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
    if (a.seqs.rows > win_of(NP)) {  // one window: nothing to hand over
        if constexpr (NP == 2)
            e = launch_local<T, 8, 1, win_of(NP)>(b, stream);
        else
            e = launch_local<T, 16, NP / 4, win_of(NP)>(b, stream);
        if (e != cudaSuccess) return e;
    }
    if (a.nchunks > 1) {
        scan_bwd_carry_kernel<<<dim3((unsigned)ceil_div((int64_t)a.ch * a.N, 256), 2), 256, 0, stream>>>(b);
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

// Chunks: so many that the third kernel's blocks fill the GPU's slots (four blocks per SM, which is what fits
// up to 16 states) kTurns times, of at least a window. 2 x 4096 tokens of 4096 channels: 1096 us with two
// turns, 1117 with three, 1087 with five, 1072 with eight (the last blocks end closer together; more
// chunks cost little).
constexpr int kTurns = 8;
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
    const int64_t n = kTurns * 4 * sms / nblk;
    q.chunk = ceil_div(ceil_div(q.rows > 0 ? q.rows : 1, n < 1 ? 1 : n), 32) * 32;
    q.nchunks = ceil_div(q.rows, q.chunk);
    if (q.nchunks < 1) q.nchunks = 1;
    q.windows = ceil_div(q.rows, win_of(np_of(p.N)));
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
