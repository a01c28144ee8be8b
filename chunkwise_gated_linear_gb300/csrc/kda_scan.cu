// Selective state space scan (kda_mixer.h: kda_scan_fwd, kda_scan_step).
//
//   h_t[n] = exp(delta_t A[n]) h_{t-1}[n] + delta_t u_t B_t[n],   y_t = sum_n C_t[n] h_t[n]
//
// per channel, so T x channels x N elements, each an exponential, two products and two
// multiply-adds. No matrix product is hidden in it: the decay differs for every (t, channel,
// state). An SM does 32 exponentials and 128 fp32 multiply-adds per clock (measured), so both pipes
// allow 32 elements per clock and SM; issuing an instruction per warp and clock on each of its
// four schedulers allows 128 / (instructions per element). The layout is chosen for few
// instructions and little shared-memory traffic per element:
//   - a thread owns two neighbouring channels and up to 16 states of each in registers. B_t and C_t,
//     the same for all channels of a group, come from shared memory once for 32 elements: 4
//     bytes per element where the SM delivers 128 bytes per clock. (One channel and four states per
//     thread, its predecessor, took 12 bytes per element and was bound by that at a third of the speed.)
//   - no exchange between lanes up to 16 states; 17 to 64 states take 2 or 4 lanes per pair of channels;
//   - fp32 pairs: two products or multiply-adds per instruction;
//   - u, dt, z are read from memory by the thread that needs them (a warp reads whole 128-byte rows), four
//     tokens ahead, and y is written from registers.
// That is parallel only over channels and sequences. Where these do not fill the GPU, the rows are
// cut into chunks: every chunk's end state from a zero start is computed (kSummary), the chunks'
// start states follow from
//   h_in[c + 1] = exp(A sum delta) h_in[c] + h_end[c]
// (scan_carry_kernel), and every chunk is walked again with its start state (kChunk). The first
// walk costs about 0.7 of the second. Bound by issue and the fp32 pipes: 4.8 and 7.0 instructions per element, 0.55
// per clock and scheduler. 2 x 8192 tokens of 4096 channels, 16 states, bf16: 526 us (2.0e12 elements/s).
#include "scan_common.cuh"

namespace kda {
namespace scan {

namespace {

enum Mode { kWhole, kSummary, kChunk };

constexpr int kFThr = 128;      // threads per block
constexpr int kTile = 32;       // tokens of B and C in shared memory
// Blocks per SM: 128 registers per thread. 2 x 8192 tokens, 4096 channels, 16 states, bf16: 525 us,
// with three blocks (168 registers) 533 us, with two 589 us.
constexpr int kPerSM = 4;
// Rows per chunk at least: 333 tokens of 2048 channels take 36 us with 16 rows (35 with 12), 48 us with
// 32, 77 us with 64 (chunks are walked serially, and there are few).
constexpr int kMinChunk = 16;
// Blocks per SM of the step kernel: two, with 128 registers, hold a sequence's states, the next one's and its
// inputs (256 sequences of 4096 x 16 states: 31 us; three blocks spill: 46; one sequence per block: 46).
constexpr int kStepPerSM = 2;

// NS states per thread, LN lanes per pair of channels.
template <int NS, int LN>
struct FwdShape {
    static constexpr int kNT = NS * LN;                 // states held per channel
    static constexpr int kChan = 2 * kFThr / LN;        // channels per block
    static constexpr int kBC = 2 * kTile * kNT / kFThr; // B and C elements per thread and tile
};

template <typename T, int NS, int LN, Mode MODE>
__global__ void __launch_bounds__(kFThr, kPerSM) scan_fwd_kernel(const ScanArgs a) {
    using S = FwdShape<NS, LN>;
    constexpr bool kOut = MODE != kSummary;
    constexpr int P2 = NS / 2;
    __shared__ __align__(16) float sB[kTile * S::kNT];
    __shared__ __align__(16) float sC[kOut ? kTile * S::kNT : 4];

    const int tid = threadIdx.x;
    const int nblk = a.G * a.blocks_per_group;
    const int blk = blockIdx.x % nblk;
    const int64_t part = blockIdx.x / nblk;  // sequence or chunk
    if (blockIdx.x == 0 && MODE != kSummary) seq_check(a.seqs, a.err, tid, kFThr);

    const int g = blk / a.blocks_per_group;
    const int first = (blk % a.blocks_per_group) * S::kChan + 2 * (tid / LN);  // within the group
    const int n0 = (tid % LN) * NS;
    // without a sign: a row's place is the same for all threads, and the thread's own part of an address then
    // needs no 64-bit arithmetic
    const uint32_t d = g * a.chg + first;
    const int nch = a.chg - first < 2 ? (a.chg - first > 0 ? 1 : 0) : 2;  // channels that exist: 0, 1, 2
    const int64_t cn = (int64_t)a.ch * a.N;
    const int64_t dn0 = (int64_t)d * a.N, dn1 = dn0 + a.N;
    const bool vst = a.vec_states && a.N == S::kNT;

    // rows of this block and the state it starts from
    int64_t c0, c1;
    SeqAt at{};
    if (MODE == kWhole) {
        if (a.seqs.cu == nullptr) {
            c0 = part * a.seqs.T;
            c1 = c0 + a.seqs.T;
        } else {
            c0 = a.seqs.cu[part];
            c1 = a.seqs.cu[part + 1];
            if (c0 < 0 || c1 < c0 || c1 > a.seqs.rows) return;  // the first block raises the error
        }
        at = SeqAt{(int)part, c0, c1};
    } else {
        c0 = part * a.chunk;
        c1 = c0 + a.chunk < a.seqs.rows ? c0 + a.chunk : a.seqs.rows;
        if (c0 < c1) at = seq_find(a.seqs, c0);
        // empty sequences keep their state; the chunks share them out
        if (MODE == kChunk && a.ht != nullptr)
            for (int64_t s = part; s < a.seqs.N; s += a.nchunks)
                if (seq_empty(a.seqs, (int)s))
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        f2 keep[P2];
                        get_states<NS>(keep, a.h0, s * cn + (r ? dn1 : dn0), n0, a.N, r < nch && a.h0 != nullptr, vst);
                        put_states<NS>(keep, a.ht, s * cn + (r ? dn1 : dn0), n0, a.N, r < nch, vst);
                    }
        if (c0 >= c1) return;
    }
    f2 h[2][P2], A2[2][P2];
    auto start = [&](const float *base, int64_t s) {
        get_states<NS>(h[0], base, s * cn + dn0, n0, a.N, nch > 0 && base != nullptr, vst);
        get_states<NS>(h[1], base, s * cn + dn1, n0, a.N, nch > 1 && base != nullptr, vst);
    };
    auto finish = [&](float *base, int64_t s) {
        put_states<NS>(h[0], base, s * cn + dn0, n0, a.N, nch > 0, vst);
        put_states<NS>(h[1], base, s * cn + dn1, n0, a.N, nch > 1, vst);
    };
    if (c0 == at.start)
        start(a.h0, at.s);
    else
        start(MODE == kChunk ? a.hchunk : nullptr, part);
    get_states<NS>(A2[0], a.A, dn0, n0, a.N, nch > 0, vst);
    get_states<NS>(A2[1], a.A, dn1, n0, a.N, nch > 1, vst);
#pragma unroll
    for (int i = 0; i < P2; ++i) {
        A2[0][i] = mul2(A2[0][i], pk(kLog2e, kLog2e));
        A2[1][i] = mul2(A2[1][i], pk(kLog2e, kLog2e));
    }
    auto two = [&](const float *p) {
        return pk(p != nullptr && nch > 0 ? p[d] : 0.f, p != nullptr && nch > 1 ? p[d + 1] : 0.f);
    };
    float bias0, bias1;
    upk(two(a.bias), bias0, bias1);
    float D0, D1;
    upk(two(kOut ? a.D : nullptr), D0, D1);
    const bool gate = kOut && a.z != nullptr;

    // four tokens of this thread's channels, read ahead; a row's place is the same for all threads
    Raw<T, 2> nu[4], ndt[4], nz[4];
    auto fetch = [&](int64_t r0) {
        const T *pu = static_cast<const T *>(a.u) + r0 * a.us;
        const T *pd = static_cast<const T *>(a.dt) + r0 * a.dts;
        const T *pz = static_cast<const T *>(a.z) + r0 * a.zs;
        if (r0 + 4 <= c1 && a.vec && nch == 2) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                nu[k].load(pu + k * a.us + d);
                ndt[k].load(pd + k * a.dts + d);
                if (gate) nz[k].load(pz + k * a.zs + d);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int n = r0 + k < c1 ? nch : 0;
                nu[k].load_some(pu + k * a.us + d, n);
                ndt[k].load_some(pd + k * a.dts + d, n);
                if (gate) nz[k].load_some(pz + k * a.zs + d, n);
            }
        }
    };
    float nbc[S::kBC];
    auto fetch_bc = [&](int64_t t0) {
#pragma unroll
        for (int k = 0; k < S::kBC; ++k) {
            const bool isC = k >= S::kBC / 2;  // the first half of the elements is B
            const int e = (tid + k * kFThr) % (kTile * S::kNT);
            const int64_t r = t0 + e / S::kNT;
            const int n = e % S::kNT;
            nbc[k] = r < c1 && n < a.N && (!isC || kOut)
                         ? to_f(static_cast<const T *>(isC ? a.C : a.B)[r * (isC ? a.cs : a.bs) + (int64_t)g * a.N + n])
                         : 0.f;
        }
    };
    float sum0 = 0.f, sum1 = 0.f;
    // one token: t in the tile, row r
    auto token = [&](int t, int64_t r, const Raw<T, 2> &ru, const Raw<T, 2> &rdt, const Raw<T, 2> &rz) {
        const float u0 = ru.get(0), u1 = ru.get(1);
        const float d0 = step_of<T>(rdt.get(0) + bias0, a.softplus), d1 = step_of<T>(rdt.get(1) + bias1, a.softplus);
        const float x0 = d0 * u0, x1 = d1 * u1;
        const f2 dd0 = pk(d0, d0), dd1 = pk(d1, d1), xx0 = pk(x0, x0), xx1 = pk(x1, x1);
        if (MODE == kSummary) {
            sum0 += d0;
            sum1 += d1;
        }
        f2 y0 = 0, y1 = 0;
#pragma unroll
        for (int i = 0; i < P2; i += 2) {
            const ulonglong2 B = *reinterpret_cast<const ulonglong2 *>(&sB[t * S::kNT + n0 + 2 * i]);
            h[0][i] = fma2(decay2(dd0, A2[0][i]), h[0][i], mul2(xx0, B.x));
            h[0][i + 1] = fma2(decay2(dd0, A2[0][i + 1]), h[0][i + 1], mul2(xx0, B.y));
            h[1][i] = fma2(decay2(dd1, A2[1][i]), h[1][i], mul2(xx1, B.x));
            h[1][i + 1] = fma2(decay2(dd1, A2[1][i + 1]), h[1][i + 1], mul2(xx1, B.y));
            if (kOut) {
                const ulonglong2 C = *reinterpret_cast<const ulonglong2 *>(&sC[t * S::kNT + n0 + 2 * i]);
                y0 = i == 0 ? mul2(h[0][0], C.x) : fma2(h[0][i], C.x, y0);
                y0 = fma2(h[0][i + 1], C.y, y0);
                y1 = i == 0 ? mul2(h[1][0], C.x) : fma2(h[1][i], C.x, y1);
                y1 = fma2(h[1][i + 1], C.y, y1);
            }
        }
        if (kOut) {
            float s0 = hsum2(y0), s1 = hsum2(y1);
#pragma unroll
            for (int o = 1; o < LN; o *= 2) {
                s0 += __shfl_xor_sync(0xffffffffu, s0, o);
                s1 += __shfl_xor_sync(0xffffffffu, s1, o);
            }
            float f[2] = {fmaf(D0, u0, s0), fmaf(D1, u1, s1)};
            if (gate) {
                f[0] *= act_value(rz.get(0), true);
                f[1] *= act_value(rz.get(1), true);
            }
            if (LN == 1 || tid % LN == 0) {
                Raw<T, 2> w;
                w.pack(f);
                T *py = static_cast<T *>(a.y) + r * a.ch;  // the same for all threads
                if (a.vec && nch == 2)
                    w.store(py + d);
                else
                    w.store_some(py + d, nch);
            }
        }
    };

    if (c0 < c1) {
        fetch(c0);
        fetch_bc(c0);
    }
    for (int64_t t0 = c0; t0 < c1; t0 += kTile) {
        __syncthreads();  // the previous tile has been read
#pragma unroll
        for (int k = 0; k < S::kBC; ++k) {
            const int e = (tid + k * kFThr) % (kTile * S::kNT);
            if (k < S::kBC / 2)
                sB[e] = nbc[k];
            else if (kOut)
                sC[e] = nbc[k];
        }
        __syncthreads();
        if (t0 + kTile < c1) fetch_bc(t0 + kTile);
#pragma unroll 1
        for (int t = 0; t < kTile; t += 4) {
            const int64_t r = t0 + t;
            if (r >= c1) break;
            Raw<T, 2> cu_[4], cdt[4], cz[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                cu_[k] = nu[k];
                cdt[k] = ndt[k];
                cz[k] = nz[k];
            }
            if (r + 4 < c1) fetch(r + 4);
            if (r + 4 <= c1 && r + 4 <= at.end) {  // four tokens of one sequence
#pragma unroll
                for (int k = 0; k < 4; ++k) token(t + k, r + k, cu_[k], cdt[k], cz[k]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (r + k >= c1) break;
                    if (r + k == at.end) {
                        if (MODE == kChunk && a.ht != nullptr) finish(a.ht, at.s);
                        seq_next(a.seqs, at);
                        start(a.h0, at.s);
                    }
                    token(t + k, r + k, cu_[k], cdt[k], cz[k]);
                }
            }
        }
    }
    if (MODE == kSummary) {
        finish(a.hchunk, part);
        if (tid % LN == 0) {
            if (nch > 0) a.schunk[part * a.ch + d] = sum0;
            if (nch > 1) a.schunk[part * a.ch + d + 1] = sum1;
        }
    } else if (a.ht != nullptr && c1 == at.end) {
        finish(a.ht, at.s);
    }
}

__global__ void __launch_bounds__(256) scan_carry_kernel(const ScanArgs a) { carry_states(a); }

// The next T tokens of each sequence. Four lanes share four channels: each lane holds a quarter of the
// states of all four (a warp reads 512 contiguous bytes of states at a time, four such reads in flight
// per thread), prepares the step size and the gate of one of them and passes the step size on to
// the others; the four outputs are added across the lanes so that each lane ends with its own
// channel's. A block goes through several sequences with the same channels, the next one's states on their
// way meanwhile. Bound by reading and writing the states (8 bytes per state; the rest is 1 / 16 of that).
template <typename T, int NP>
__global__ void __launch_bounds__(256, NP <= 4 ? kStepPerSM : 1) scan_step_kernel(const ScanArgs a) {
    const uint32_t tid = threadIdx.x, lane = tid & 31, nl = tid & 3, n0 = nl * NP;
    // places are a part that is the same for the block and the thread's own, in 32 bits without a sign
    const uint32_t nblk = (a.ch + 255u) / 256u, blk = blockIdx.x % nblk;
    const int per = gridDim.x / nblk;  // blocks that share the sequences
    const uint32_t base = blk * 256 + (tid >> 5) * 32 + (lane >> 2), ch = a.ch, N = a.N;
    const uint32_t own = base + nl * 8;  // the channel that this lane prepares and finishes
    const bool live = own < ch;
    const bool full = a.vec_states && N == 4 * NP && blk * 256 + 256 <= ch;  // whole vectors, all of them
    const bool one_group = a.G == 1 || a.chg % 32 == 0;                      // of a warp's 32 channels
    float next[4][NP], A2[4][NP];  // the states of the sequence whose turn is next
    auto load = [&](float (&h)[4][NP], const float *from) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint32_t d = base + r * 8;
            if (full)
                load_vec<float, NP>(h[r], from + (d * N + n0));
            else
                load_states<NP>(h[r], from, d * N, nl, N, d < ch);
        }
    };
    int64_t seq = blockIdx.x / nblk;
    constexpr bool kNext = NP <= 8;  // registers for the next sequence's states
    if (kNext) load(next, a.h0 + seq * ch * N);
    load(A2, a.A);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < NP; ++i) A2[r][i] *= kLog2e;
    const float bias = a.bias != nullptr && live ? a.bias[own] : 0.f, D = a.D != nullptr && live ? a.D[own] : 0.f;
    float B[NP], C[NP];
    auto load_bc = [&](const T *pB, const T *pC, uint32_t d) {  // of channel d's group
        const uint32_t o = (a.G == 1 ? 0u : (d < ch ? d : ch - 1) / a.chg * N) + n0;
        if (a.vec && N == 4 * NP) {
            load_vec<T, NP>(B, pB + o);
            load_vec<T, NP>(C, pC + o);
        } else {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                B[i] = n0 + i < N ? to_f(pB[o + i]) : 0.f;
                C[i] = n0 + i < N ? to_f(pC[o + i]) : 0.f;
            }
        }
    };
    // a token's inputs, read one token ahead
    const bool ahead = one_group && a.vec && N == 4 * NP;  // B and C too
    Raw<T, 1> nu, ns, nz;
    Raw<T, NP> nB, nC;
    const uint32_t obc = (a.G == 1 ? 0u : (base < ch ? base : ch - 1) / a.chg * N) + n0;
    auto fetch = [&](int64_t row) {
        if (live) {
            nu.load(static_cast<const T *>(a.u) + row * a.us + own);
            ns.load(static_cast<const T *>(a.dt) + row * a.dts + own);
            if (a.z != nullptr) nz.load(static_cast<const T *>(a.z) + row * a.zs + own);
        }
        if (ahead) {
            nB.load(static_cast<const T *>(a.B) + row * a.bs + obc);
            nC.load(static_cast<const T *>(a.C) + row * a.cs + obc);
        }
    };
    const int T_ = a.seqs.T;
    nu.zero();
    ns.zero();
    nz.zero();
    if (T_ > 0) fetch(seq * T_);
    for (; seq < a.seqs.N; seq += per) {
        float h[4][NP];
        const bool more = seq + per < a.seqs.N;
        if constexpr (kNext) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int i = 0; i < NP; ++i) h[r][i] = next[r][i];
            if (more) load(next, a.h0 + (seq + per) * ch * N);
        } else {
            load(h, a.h0 + seq * ch * N);
        }
        for (int t = 0; t < T_; ++t) {
            const int64_t row = seq * T_ + t;
            const float u = nu.get(0), s = ns.get(0), z = nz.get(0);
            if (ahead) {
                nB.unpack(B);
                nC.unpack(C);
            } else if (one_group) {
                load_bc(static_cast<const T *>(a.B) + row * a.bs, static_cast<const T *>(a.C) + row * a.cs, base);
            }
            if (t + 1 < T_)
                fetch(row + 1);
            else if (more)
                fetch((seq + per) * T_);
            const float delta = step_of<T>(s + bias, a.softplus), x = delta * u;
            float p[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (!one_group)
                    load_bc(static_cast<const T *>(a.B) + row * a.bs, static_cast<const T *>(a.C) + row * a.cs, base + r * 8);
                const float dr = __shfl_sync(0xffffffffu, delta, (lane & ~3u) + r);
                const float xr = __shfl_sync(0xffffffffu, x, (lane & ~3u) + r);
                p[r] = 0.f;
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    h[r][i] = fmaf(tc5::ex2(fmaf(dr, A2[r][i], kExpFix)), h[r][i], xr * B[i]);
                    p[r] = fmaf(C[i], h[r][i], p[r]);
                }
            }
            float y = fmaf(D, u, sum_lanes(p, nl));
            if (a.z != nullptr) y *= act_value(z, true);
            if (live) (static_cast<T *>(a.y) + row * ch)[own] = from_f<T>(y);
        }
        float *ht = a.ht + seq * ch * N;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint32_t d = base + r * 8;
            if (full)
                store_vec<float, NP>(ht + (d * N + n0), h[r]);
            else
                store_states<NP>(h[r], ht, d * N, nl, N, d < ch);
        }
    }
}

template <typename T, int NS, int LN, Mode MODE>
cudaError_t launch_shape(ScanArgs a, int64_t parts, cudaStream_t stream) {
    a.blocks_per_group = (int)ceil_div(a.chg, FwdShape<NS, LN>::kChan);
    const int64_t grid = parts * a.G * a.blocks_per_group;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    scan_fwd_kernel<T, NS, LN, MODE><<<(unsigned)grid, kFThr, 0, stream>>>(a);
    return cudaGetLastError();
}
template <typename T, Mode MODE>
cudaError_t launch_mode(const ScanArgs &a, int64_t parts, cudaStream_t stream) {
    if (a.N <= 8) return launch_shape<T, 8, 1, MODE>(a, parts, stream);
    if (a.N <= 16) return launch_shape<T, 16, 1, MODE>(a, parts, stream);
    if (a.N <= 32) return launch_shape<T, 16, 2, MODE>(a, parts, stream);
    return launch_shape<T, 16, 4, MODE>(a, parts, stream);
}
int fwd_channels(int N) { return N <= 16 ? 2 * kFThr : (N <= 32 ? kFThr : kFThr / 2); }

template <typename T>
cudaError_t launch_step(const ScanArgs &a, cudaStream_t stream) {
    // the blocks of 256 channels, each as often as fills the GPU's slots once
    const int64_t nblk = ceil_div(a.ch, 256);
    int64_t per = (int64_t)kStepPerSM * (sm_count() > 0 ? sm_count() : 1) / nblk;
    per = per < 1 ? 1 : (per > a.seqs.N ? a.seqs.N : per);
    const int64_t grid = per * nblk;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    switch (np_of(a.N)) {
        case 2:
            scan_step_kernel<T, 2><<<(unsigned)grid, 256, 0, stream>>>(a);
            break;
        case 4:
            scan_step_kernel<T, 4><<<(unsigned)grid, 256, 0, stream>>>(a);
            break;
        case 8:
            scan_step_kernel<T, 8><<<(unsigned)grid, 256, 0, stream>>>(a);
            break;
        default:
            scan_step_kernel<T, 16><<<(unsigned)grid, 256, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

int elem_size(int dtype) { return dtype == KDA_DTYPE_BF16 ? 2 : 4; }

// Chunks of the forward pass: none (0) where one block per sequence and block of channels gives
// three blocks per SM, else as many as fill the GPU's slots (kPerSM blocks per SM) once.
struct FwdPlan {
    int64_t chunk, nchunks;
    size_t bytes;
};
FwdPlan fwd_plan(const kda_scan_params &p) {
    FwdPlan q{};
    const int64_t rows = p.cu_seqlens != nullptr ? (int64_t)p.T : (int64_t)p.batch * p.T;
    const int64_t nblk = (int64_t)p.G * ceil_div(p.channels / p.G, fwd_channels(p.N));
    const int64_t sms = sm_count() > 0 ? sm_count() : 1;
    const bool ragged = p.cu_seqlens != nullptr && rows > 4 * (int64_t)p.batch;
    if (!ragged && nblk * p.batch >= 3 * sms) return q;
    if (!ragged && ceil_div(rows, p.batch) < 64) return q;
    int64_t n = kPerSM * sms / nblk;
    if (n < 1) n = 1;
    int64_t chunk = ceil_div(ceil_div(rows, n), 4) * 4;
    if (chunk < kMinChunk) chunk = kMinChunk;
    if (chunk >= rows && !ragged) return q;
    q.chunk = chunk;
    q.nchunks = ceil_div(rows, chunk);
    q.bytes = (size_t)q.nchunks * p.channels * (p.N + 1) * sizeof(float);
    return q;
}

template <typename T>
cudaError_t run_fwd(const ScanArgs &a, cudaStream_t stream) {
    if (a.nchunks == 0) return launch_mode<T, kWhole>(a, a.seqs.N, stream);
    cudaError_t e = cudaSuccess;
    if (a.nchunks > 1) e = launch_mode<T, kSummary>(a, a.nchunks - 1, stream);  // nothing follows the last
    if (e == cudaSuccess && a.nchunks > 1) {
        scan_carry_kernel<<<(unsigned)ceil_div((int64_t)a.ch * a.N, 256), 256, 0, stream>>>(a);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) e = launch_mode<T, kChunk>(a, a.nchunks, stream);
    return e;
}

}  // namespace

int scan_check(const kda_scan_params &p) {
    if (p.batch < 1 || p.T < 0 || p.channels < 1 || p.N < 1 || p.G < 1 || p.channels % p.G != 0) return KDA_ERR_INVALID_ARG;
    const int64_t bc = (int64_t)p.G * p.N;
    const int64_t strides[] = {p.u_stride, p.dt_stride, p.z_stride, p.B_stride, p.C_stride};
    for (int i = 0; i < 5; ++i)
        if (strides[i] < 0 || (strides[i] != 0 && strides[i] < (i < 3 ? (int64_t)p.channels : bc))) return KDA_ERR_INVALID_ARG;
    if (p.A == nullptr || (p.T != 0 && (p.u == nullptr || p.dt == nullptr || p.B == nullptr || p.C == nullptr)))
        return KDA_ERR_INVALID_ARG;
    if (p.dtype != KDA_DTYPE_BF16 && p.dtype != KDA_DTYPE_F32) return KDA_ERR_UNSUPPORTED;
    if (p.N > kMaxN) return KDA_ERR_UNSUPPORTED;
    const int e = elem_size(p.dtype);
    if (!aligned(p.u, e) || !aligned(p.dt, e) || !aligned(p.B, e) || !aligned(p.C, e) || !aligned(p.z, e)) return KDA_ERR_ALIGNMENT;
    if (!aligned(p.A, 4) || !aligned(p.D, 4) || !aligned(p.dt_bias, 4) || !aligned(p.h0, 4) || !aligned(p.cu_seqlens, 4))
        return KDA_ERR_ALIGNMENT;
    const int64_t rows = p.cu_seqlens != nullptr ? (int64_t)p.T : (int64_t)p.batch * p.T;
    if (rows > INT32_MAX || bc > INT32_MAX || (int64_t)p.channels * p.N > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

ScanArgs scan_args(const kda_scan_params &p, const void *const *more, int n) {
    ScanArgs a{};
    a.u = p.u;
    a.dt = p.dt;
    a.A = p.A;
    a.B = p.B;
    a.C = p.C;
    a.D = p.D;
    a.z = p.z;
    a.bias = p.dt_bias;
    a.h0 = p.h0;
    a.us = p.u_stride != 0 ? p.u_stride : p.channels;
    a.dts = p.dt_stride != 0 ? p.dt_stride : p.channels;
    a.zs = p.z_stride != 0 ? p.z_stride : p.channels;
    a.bs = p.B_stride != 0 ? p.B_stride : (int64_t)p.G * p.N;
    a.cs = p.C_stride != 0 ? p.C_stride : (int64_t)p.G * p.N;
    a.ch = p.channels;
    a.N = p.N;
    a.G = p.G;
    a.chg = p.channels / p.G;
    a.blocks_per_group = (int)ceil_div(a.chg, kDB);
    a.softplus = p.dt_softplus != 0;
    const int per16 = 16 / elem_size(p.dtype);
    bool vec = a.us % per16 == 0 && a.dts % per16 == 0 && (p.z == nullptr || a.zs % per16 == 0) && a.ch % 8 == 0 &&
               a.chg % 8 == 0 && aligned(p.u, 16) && aligned(p.dt, 16) && aligned(p.z, 16);
    for (int i = 0; i < n; ++i) vec = vec && aligned(more[i], 16);
    a.vec = vec;
    a.seqs = Seqs{p.cu_seqlens, p.batch, p.T, p.cu_seqlens != nullptr ? (int64_t)p.T : (int64_t)p.batch * p.T};
    return a;
}

namespace {

int fwd_check(const kda_scan_params &p) {
    const int st = scan_check(p);
    if (st != KDA_OK) return st;
    if (p.T != 0 && p.y == nullptr) return KDA_ERR_INVALID_ARG;
    if (!aligned(p.y, elem_size(p.dtype)) || !aligned(p.ht, 4)) return KDA_ERR_ALIGNMENT;
    return KDA_OK;
}

}  // namespace
}  // namespace scan
}  // namespace kda

extern "C" {

size_t kda_scan_fwd_workspace(const kda_scan_params *p) {
    using namespace kda::scan;
    return p == nullptr || fwd_check(*p) != KDA_OK ? 0 : fwd_plan(*p).bytes;
}

int kda_scan_fwd(const kda_scan_params *p, cudaStream_t stream) {
    using namespace kda;
    using namespace kda::scan;
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    const int st = fwd_check(*p);
    if (st != KDA_OK) return st;
    // chunks read h0 while others have already written ht
    if (p->ht != nullptr && p->ht == p->h0) return KDA_ERR_INVALID_ARG;
    const FwdPlan q = fwd_plan(*p);
    if (p->workspace != nullptr && p->workspace_bytes < q.bytes) return KDA_ERR_INVALID_ARG;
    if (!aligned(p->workspace, 16)) return KDA_ERR_ALIGNMENT;
    ScanArgs a = scan_args(*p, nullptr, 0);
    a.y = p->y;
    a.ht = p->ht;
    a.chunk = q.chunk;
    a.nchunks = q.nchunks;
    cudaError_t e = device_error_word(&a.err);
    if (e != cudaSuccess) return status_of_cuda(e);
    Scratch ws;
    e = ws.get(p->workspace, q.bytes, stream);
    if (e != cudaSuccess) return status_of_cuda(e);
    const size_t e2 = 2 * elem_size(p->dtype);  // pairs of channels
    a.vec = a.us % 2 == 0 && a.dts % 2 == 0 && (p->z == nullptr || a.zs % 2 == 0) && a.ch % 2 == 0 && a.chg % 2 == 0 &&
            aligned(p->u, e2) && aligned(p->dt, e2) && aligned(p->z, e2) && aligned(p->y, e2);
    a.vec_states = aligned(p->A, 16) && aligned(p->h0, 16) && aligned(p->ht, 16) && p->N % 4 == 0;
    a.hchunk = static_cast<float *>(ws.ptr);
    a.schunk = a.hchunk + q.nchunks * (int64_t)p->channels * p->N;
    e = p->dtype == KDA_DTYPE_BF16 ? run_fwd<bf16>(a, stream) : run_fwd<float>(a, stream);
    return status_of_cuda(ws.release(e));
}

int kda_scan_step(const kda_scan_params *p, cudaStream_t stream) {
    using namespace kda;
    using namespace kda::scan;
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    const int st = fwd_check(*p);
    if (st != KDA_OK) return st;
    if (p->cu_seqlens != nullptr || p->h0 == nullptr || p->ht == nullptr) return KDA_ERR_INVALID_ARG;
    ScanArgs a = scan_args(*p, nullptr, 0);
    a.y = p->y;
    a.ht = p->ht;
    // B and C by the lane's quarter of the states (at most 16 bytes at a time)
    const int np = np_of(p->N), e = elem_size(p->dtype);
    const int span = np * e > 16 ? 16 : np * e;
    a.vec = a.bs * e % span == 0 && a.cs * e % span == 0 && aligned(p->B, span) && aligned(p->C, span);
    a.vec_states = aligned(p->A, 16) && aligned(p->h0, 16) && aligned(p->ht, 16);
    return status_of_cuda(p->dtype == KDA_DTYPE_BF16 ? launch_step<bf16>(a, stream) : launch_step<float>(a, stream));
}

}  // extern "C"
