// Selective state space scan (kda_mixer.h: kda_scan_fwd, kda_scan_step).
//
//   h_t[n] = exp(delta_t A[n]) h_{t-1}[n] + delta_t u_t B_t[n],   y_t = sum_n C_t[n] h_t[n]
//
// per channel, so T x channels x N elements, each an exponential, two products and two
// multiply-adds. No matrix product is hidden in it: the decay differs for every (t, channel,
// state). On this GPU an SM does 32 exponentials and 128 fp32 multiply-adds per clock, so both
// pipes allow 32 elements per clock and SM; reading u, dt, z and writing y takes
// about as long (N = 16, bf16). The kernels are built to keep both pipes fed:
//   - states stay in registers, four lanes per channel (enough threads without cutting T);
//   - fp32 pairs: two products or multiply-adds per instruction;
//   - tiles of 32 tokens: step sizes and u are prepared once per (token, channel) by 16-byte
//     vectors and handed over in shared memory, the next tile's loads are in flight meanwhile;
//   - the sum over the states of four steps takes three exchanges between lanes.
// Where channels x sequences fill the GPU, a block walks its sequence from start to end. Where
// they do not, the rows are cut into chunks: every chunk's end state from a zero start is computed
// (kSummary), the chunks' start states follow from
//   h_in[c + 1] = exp(A sum delta) h_in[c] + h_end[c]
// (scan_carry_kernel), and every chunk is walked again with its start state (kChunk). The first
// walk costs about 0.6 of the second.
#include "scan_common.cuh"

namespace kda {
namespace scan {

namespace {

enum Mode { kWhole, kSummary, kChunk };

// Steps t0 .. t0 + 3 of a tile for this thread's channel and states.
template <int NP, bool OUT>
__device__ __forceinline__ void step4(f2 (&h)[NP / 2], const f2 (&A)[NP / 2], const float4 (*sx)[kDB], const float *sB,
                                      const float *sC, int nt, int t0, int slot, int nl, float (&p)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int t = t0 + k;
        const ulonglong2 dx = *reinterpret_cast<const ulonglong2 *>(&sx[t][slot]);  // (delta, delta), (delta u, delta u)
        f2 B[NP / 2], C[NP / 2];
        lds_pairs<NP>(B, sB + t * nt + nl * NP);
        if (OUT) lds_pairs<NP>(C, sC + t * nt + nl * NP);
        f2 s = 0;
#pragma unroll
        for (int i = 0; i < NP / 2; ++i) {
            h[i] = fma2(exp2_2(mul2(dx.x, A[i])), h[i], mul2(dx.y, B[i]));
            if (OUT) s = i == 0 ? mul2(h[0], C[0]) : fma2(h[i], C[i], s);
        }
        if (OUT) p[k] = hsum2(s);
    }
}

template <typename T, int NP, Mode MODE>
__global__ void __launch_bounds__(kThreads) scan_fwd_kernel(const ScanArgs a) {
    constexpr bool kOut = MODE != kSummary;
    constexpr int kNT = kLN * NP;                      // states per channel held
    constexpr int kBC = 2 * kTK * kNT / kThreads;      // B and C elements per thread and tile
    constexpr int kYRow = kDB + 8;                     // padded: four steps x eight channels hit 32 banks
    __shared__ __align__(16) float4 sx[kTK][kDB];
    __shared__ __align__(16) float sB[kTK * kNT];
    __shared__ __align__(16) float sC[kOut ? kTK * kNT : 4];
    __shared__ __align__(16) float sy[kOut ? kTK : 1][kYRow];

    const int tid = threadIdx.x;
    const int nblk = a.G * a.blocks_per_group;
    const Chans ch = chans_of(a, blockIdx.x % nblk);
    const int64_t part = blockIdx.x / nblk;  // sequence or chunk
    if (blockIdx.x == 0 && MODE != kSummary) seq_check(a.seqs, a.err, tid, kThreads);

    const int dl = tid >> 2, nl = tid & 3, slot = slot_of(dl);
    const int d = ch.d0 + dl;
    const bool live = dl < ch.n;
    const int64_t dn = (int64_t)d * a.N;

    // rows of this block and the state it starts from
    int64_t c0, c1;
    SeqAt at;
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
                if (seq_empty(a.seqs, (int)s)) {
                    float keep[NP];
                    load_states<NP>(keep, a.h0, s * a.ch * a.N + dn, nl, a.N, live && a.h0 != nullptr);
                    store_states<NP>(keep, a.ht, s * a.ch * a.N + dn, nl, a.N, live);
                }
        if (c0 >= c1) return;
    }
    float h[NP], An[NP];
    if (c0 == at.start)
        load_states<NP>(h, a.h0, (int64_t)at.s * a.ch * a.N + dn, nl, a.N, live && a.h0 != nullptr);
    else
        load_states<NP>(h, a.hchunk, part * a.ch * a.N + dn, nl, a.N, live && MODE == kChunk);
    load_states<NP>(An, a.A, dn, nl, a.N, live);
#pragma unroll
    for (int i = 0; i < NP; ++i) An[i] *= kLog2e;
    f2 hp[NP / 2], A2[NP / 2];
    to_pairs<NP>(hp, h);
    to_pairs<NP>(A2, An);

    // staging: token tr of a tile, channels 8 tc .. 8 tc + 7 of the block
    const int tr = tid >> 3, tc = (tid & 7) * 8;
    const int nc = ch.n - tc;  // channels that exist here (may be <= 0)
    const int64_t dc = ch.d0 + tc;
    float bias8[8], D8[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        bias8[j] = a.bias != nullptr && j < nc ? a.bias[dc + j] : 0.f;
        D8[j] = kOut && a.D != nullptr && j < nc ? a.D[dc + j] : 0.f;
    }
    Raw<T, 8> nu, ndt, nz;
    float nbc[kBC];
    auto fetch = [&](int64_t t0) {
        const int64_t r = t0 + tr;
        const int n = r < c1 ? nc : 0;
        load8<T>(nu, a.u, r * a.us + dc, n, a.vec);
        load8<T>(ndt, a.dt, r * a.dts + dc, n, a.vec);
        if (kOut && a.z != nullptr) load8<T>(nz, a.z, r * a.zs + dc, n, a.vec);
#pragma unroll
        for (int k = 0; k < kBC; ++k) {
            const int e = (tid + k * kThreads) % (kTK * kNT);
            const bool isC = k >= kBC / 2;  // the first half of the elements is B
            const int64_t rr = t0 + e / kNT;
            const int n2 = e % kNT;
            float v = 0.f;
            if (rr < c1 && n2 < a.N && (!isC || kOut)) {
                const void *src = isC ? a.C : a.B;
                v = to_f(static_cast<const T *>(src)[rr * (isC ? a.cs : a.bs) + (int64_t)ch.g * a.N + n2]);
            }
            nbc[k] = v;
        }
    };
    float sum_delta[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sum_delta[j] = 0.f;

    if (c0 < c1) fetch(c0);
    for (int64_t t0 = c0; t0 < c1; t0 += kTK) {
        Raw<T, 8> cu_ = nu, cz = nz;
        __syncthreads();  // the previous tile has been read
        {
            const bool row = t0 + tr < c1;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // rows past the end: no step, the state stays
                const float delta = row && j < nc ? step_of<T>(ndt.get(j) + bias8[j], a.softplus) : 0.f;
                const float x = delta * cu_.get(j);
                sx[tr][slot_of(tc + j)] = make_float4(delta, delta, x, x);
                if (MODE == kSummary) sum_delta[j] += delta;
            }
#pragma unroll
            for (int k = 0; k < kBC; ++k) {
                const int e = (tid + k * kThreads) % (kTK * kNT);
                if (k < kBC / 2)
                    sB[e] = nbc[k];
                else if (kOut)
                    sC[e] = nbc[k];
            }
        }
        __syncthreads();
        if (t0 + kTK < c1) fetch(t0 + kTK);

        const int64_t tile_end = t0 + kTK < c1 ? t0 + kTK : c1;
        if (at.end >= tile_end) {  // one sequence in the whole tile
#pragma unroll 2
            for (int t = 0; t < kTK; t += 4) {
                float p[4];
                step4<NP, kOut>(hp, A2, sx, sB, sC, kNT, t, slot, nl, p);
                if (kOut) sy[t + nl][dl] = sum_lanes(p, nl);
            }
        } else {  // sequences end inside the tile: token by token
            for (int t = 0; t < (int)(tile_end - t0); ++t) {
                if (t0 + t == at.end) {
                    if (MODE == kChunk && a.ht != nullptr) {
                        from_pairs<NP>(h, hp);
                        store_states<NP>(h, a.ht, (int64_t)at.s * a.ch * a.N + dn, nl, a.N, live);
                    }
                    seq_next(a.seqs, at);
                    load_states<NP>(h, a.h0, (int64_t)at.s * a.ch * a.N + dn, nl, a.N, live && a.h0 != nullptr);
                    to_pairs<NP>(hp, h);
                }
                const ulonglong2 dx = *reinterpret_cast<const ulonglong2 *>(&sx[t][slot]);
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < NP / 2; ++i) {
                    const f2 B = *reinterpret_cast<const f2 *>(&sB[t * kNT + nl * NP + 2 * i]);
                    hp[i] = fma2(exp2_2(mul2(dx.x, A2[i])), hp[i], mul2(dx.y, B));
                    if (kOut) s += hsum2(mul2(hp[i], *reinterpret_cast<const f2 *>(&sC[t * kNT + nl * NP + 2 * i])));
                }
                if (kOut) {
                    s += __shfl_xor_sync(0xffffffffu, s, 1);
                    s += __shfl_xor_sync(0xffffffffu, s, 2);
                    if (nl == 0) sy[t][dl] = s;
                }
            }
        }
        if (kOut) {
            __syncthreads();
            const int64_t r = t0 + tr;
            if (r < c1 && nc > 0) {
                float out[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    out[j] = fmaf(D8[j], cu_.get(j), sy[tr][tc + j]);
                    if (a.z != nullptr) out[j] *= act_value(cz.get(j), true);
                }
                store8<T>(a.y, r * a.ch + dc, out, nc, a.vec);
            }
        }
    }
    from_pairs<NP>(h, hp);
    if (MODE == kSummary) {
        store_states<NP>(h, a.hchunk, part * a.ch * a.N + dn, nl, a.N, live);
        // sum of the step sizes over the 32 token rows of the staging threads, in a fixed order
        __syncthreads();
        float *red = reinterpret_cast<float *>(&sx[0][0]);  // [32][64]
#pragma unroll
        for (int j = 0; j < 8; ++j) red[tr * kDB + tc + j] = sum_delta[j];
        __syncthreads();
        if (tid < ch.n) {
            float s = 0.f;
            for (int i = 0; i < kTK; ++i) s += red[i * kDB + tid];
            a.schunk[part * a.ch + ch.d0 + tid] = s;
        }
    } else if (a.ht != nullptr && c1 == at.end) {
        store_states<NP>(h, a.ht, (int64_t)at.s * a.ch * a.N + dn, nl, a.N, live);
    }
}

// Chunk end states to chunk start states, in place; one thread per (channel, state) walks
// the chunks, eight loads ahead. A chunk in which a sequence starts does not pass its start
// state on. Chunk 0 starts a sequence: its own start state is not read.
__global__ void __launch_bounds__(256) scan_carry_kernel(const ScanArgs a) {
    constexpr int kAhead = 8;
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

// The next T tokens of each sequence: 4 lanes per channel as above, no tiles. Bound by
// reading and writing the states (8 bytes per state; everything else is 1 / 16 of that).
template <typename T, int NP>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(const ScanArgs a) {
    const int tid = threadIdx.x, nl = tid & 3;
    const int nblk = (a.ch + kDB - 1) / kDB;
    const int64_t seq = blockIdx.x / nblk;
    const int d = (int)(blockIdx.x % nblk) * kDB + (tid >> 2);
    const bool live = d < a.ch;
    const int dd = live ? d : a.ch - 1;  // every lane takes part in the exchanges
    const int64_t at = (seq * a.ch + dd) * a.N;
    float h[NP], An[NP];
    if (NP == 4 && a.N == 16 && a.vec) {  // whole vectors
        load_vec<float, NP>(h, a.h0 + at + nl * NP);
        load_vec<float, NP>(An, a.A + (int64_t)dd * a.N + nl * NP);
    } else {
        load_states<NP>(h, a.h0, at, nl, a.N, true);
        load_states<NP>(An, a.A, (int64_t)dd * a.N, nl, a.N, true);
    }
    const float bias = a.bias != nullptr ? a.bias[dd] : 0.f, D = a.D != nullptr ? a.D[dd] : 0.f;
    const int g = dd / a.chg;
    for (int t = 0; t < a.seqs.T; ++t) {
        const int64_t r = seq * a.seqs.T + t;
        const float u = to_f(static_cast<const T *>(a.u)[r * a.us + dd]);
        const float delta = step_of<T>(to_f(static_cast<const T *>(a.dt)[r * a.dts + dd]) + bias, a.softplus);
        const float x = delta * u;
        const T *B = static_cast<const T *>(a.B) + r * a.bs + (int64_t)g * a.N;
        const T *C = static_cast<const T *>(a.C) + r * a.cs + (int64_t)g * a.N;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int n = nl * NP + i;
            const bool in = n < a.N;
            const float b = in ? to_f(B[n]) : 0.f, c = in ? to_f(C[n]) : 0.f;
            h[i] = fmaf(tc5::ex2(delta * (An[i] * kLog2e)), h[i], x * b);
            s = fmaf(c, h[i], s);
        }
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        if (nl == 0 && live) {
            s = fmaf(D, u, s);
            if (a.z != nullptr) s *= act_value(to_f(static_cast<const T *>(a.z)[r * a.zs + dd]), true);
            static_cast<T *>(a.y)[r * a.ch + dd] = from_f<T>(s);
        }
    }
    if (NP == 4 && a.N == 16 && a.vec) {
        if (live) store_vec<float, NP>(a.ht + at + nl * NP, h);
    } else {
        store_states<NP>(h, a.ht, at, nl, a.N, live);
    }
}

template <typename T, Mode MODE>
cudaError_t launch_mode(const ScanArgs &a, int64_t parts, cudaStream_t stream) {
    const int64_t grid = parts * a.G * a.blocks_per_group;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    switch (np_of(a.N)) {
        case 2:
            scan_fwd_kernel<T, 2, MODE><<<(unsigned)grid, kThreads, 0, stream>>>(a);
            break;
        case 4:
            scan_fwd_kernel<T, 4, MODE><<<(unsigned)grid, kThreads, 0, stream>>>(a);
            break;
        case 8:
            scan_fwd_kernel<T, 8, MODE><<<(unsigned)grid, kThreads, 0, stream>>>(a);
            break;
        default:
            scan_fwd_kernel<T, 16, MODE><<<(unsigned)grid, kThreads, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_step(const ScanArgs &a, cudaStream_t stream) {
    const int64_t grid = (int64_t)a.seqs.N * ceil_div(a.ch, kDB);
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    switch (np_of(a.N)) {
        case 2:
            scan_step_kernel<T, 2><<<(unsigned)grid, kThreads, 0, stream>>>(a);
            break;
        case 4:
            scan_step_kernel<T, 4><<<(unsigned)grid, kThreads, 0, stream>>>(a);
            break;
        case 8:
            scan_step_kernel<T, 8><<<(unsigned)grid, kThreads, 0, stream>>>(a);
            break;
        default:
            scan_step_kernel<T, 16><<<(unsigned)grid, kThreads, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

int elem_size(int dtype) { return dtype == KDA_DTYPE_BF16 ? 2 : 4; }

// Chunks of the forward pass: none (0) where one block per sequence and 64 channels gives
// about a block per SM, else as many as give three blocks per SM, of at least 64 rows.
struct FwdPlan {
    int64_t chunk, nchunks;
    size_t bytes;
};
FwdPlan fwd_plan(const kda_scan_params &p) {
    FwdPlan q{};
    const int64_t rows = p.cu_seqlens != nullptr ? (int64_t)p.T : (int64_t)p.batch * p.T;
    const int64_t nblk = (int64_t)p.G * ceil_div(p.channels / p.G, kDB);
    const int64_t sms = sm_count() > 0 ? sm_count() : 1;
    const bool ragged = p.cu_seqlens != nullptr && rows > 4 * (int64_t)p.batch;
    if (!ragged && nblk * p.batch * 10 >= sms * 8) return q;
    const int64_t per_seq = ceil_div(rows, p.batch);
    if (!ragged && per_seq < 128) return q;
    int64_t n = ceil_div(3 * sms, nblk);
    int64_t chunk = ceil_div(ceil_div(rows, n), kTK) * kTK;
    if (chunk < 64) chunk = 64;
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
    if (e == cudaSuccess && a.nchunks > 1) e = launch_scan_carry(a, stream);
    if (e == cudaSuccess) e = launch_mode<T, kChunk>(a, a.nchunks, stream);
    return e;
}

}  // namespace

cudaError_t launch_scan_summary(const ScanArgs &a, int dtype, cudaStream_t stream) {
    if (a.nchunks <= 1) return cudaSuccess;
    return dtype == KDA_DTYPE_BF16 ? launch_mode<bf16, kSummary>(a, a.nchunks - 1, stream)
                                   : launch_mode<float, kSummary>(a, a.nchunks - 1, stream);
}

cudaError_t launch_scan_carry(const ScanArgs &a, cudaStream_t stream) {
    scan_carry_kernel<<<(unsigned)ceil_div((int64_t)a.ch * a.N, 256), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

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
    if (rows > INT32_MAX || bc > INT32_MAX) return KDA_ERR_UNSUPPORTED;
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
    const FwdPlan q = fwd_plan(*p);
    if (p->workspace != nullptr && p->workspace_bytes < q.bytes) return KDA_ERR_INVALID_ARG;
    if (!aligned(p->workspace, 16)) return KDA_ERR_ALIGNMENT;
    const void *more[] = {p->y};
    ScanArgs a = scan_args(*p, more, 1);
    a.y = p->y;
    a.ht = p->ht;
    a.chunk = q.chunk;
    a.nchunks = q.nchunks;
    cudaError_t e = device_error_word(&a.err);
    if (e != cudaSuccess) return status_of_cuda(e);
    Scratch ws;
    e = ws.get(p->workspace, q.bytes, stream);
    if (e != cudaSuccess) return status_of_cuda(e);
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
    a.vec = aligned(p->A, 16) && aligned(p->h0, 16) && aligned(p->ht, 16);  // the states and A here
    return status_of_cuda(p->dtype == KDA_DTYPE_BF16 ? launch_step<bf16>(a, stream) : launch_step<float>(a, stream));
}

}  // extern "C"
