// Attention over a paged cache (kda_attention.h): the checks and the join of the pieces of items that were cut.
#include "attn_launch.h"

namespace kda {
namespace attn {
namespace {

constexpr int kJoinWarps = 8;
constexpr int kJoinThreads = 32 * kJoinWarps;

// A query row of an item that was cut: the largest m of its pieces, then the sum of 2^(m - max) (l, O) over them. `split` warps
// share a row's pieces, every split-th each, and their sums are added in order; lane i holds channels 4 i .. 4 i + 3
// (and + 128). A block with nothing to join ends after the plan, which is made while the attention still runs.
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ Args a, int split) {
    __shared__ int64_t mem[kJoinWarps], mine;
    __shared__ float4 sums[kJoinWarps][64];
    __shared__ float ls[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x / a.per_seq, item = blockIdx.x - b * a.per_seq;
    Scan<kJoinThreads> sc;
    sc.run(a, mem);
    if (b >= sc.first && b < sc.first + sc.each) {  // one thread's
        int64_t before = sc.before;
        for (int x = sc.first; x < b; ++x) before += (int64_t)units_of(cache_len(a.cache, x), a.unit) * a.per_seq;
        mine = before;
    }
    __syncthreads();
    const int n = sharers(a, sc.total);
    const int len = cache_len(a.cache, b), units = units_of(len, a.unit);
    const int64_t begin = mine + (int64_t)item * units;
    const int w0 = owner(sc.total, begin, n), w1 = owner(sc.total, begin + units - 1, n);
    if (w0 == w1) return;
    const Piece p = piece_of(a, b, len, item, 0, units);
    const int D = a.cache.D, part = warp % split;
    const int r = blockIdx.y * (kJoinWarps / split) + warp / split;
    wait_for_previous();
    float m = -INFINITY, l = 0.f;
    float4 s[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    if (r < p.rows) {
        // the piece of the first worker begins there, the others come from the one before
        auto stats = [&](int w) { return reinterpret_cast<const float2 *>(piece_mem(a, w, w == w0) + (int64_t)a.rows * D)[r]; };
        for (int w = w0 + lane; w <= w1; w += 32) m = fmaxf(m, stats(w).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll 4
        for (int w = w0 + part; w <= w1; w += split) {
            const float2 x = stats(w);
            const float f = tc5::ex2(x.x - ref);
            l = fmaf(x.y, f, l);
            const float *from = piece_mem(a, w, w == w0) + (int64_t)r * D + 4 * lane;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (4 * lane + 128 * h < D) {
                    const float4 v = *reinterpret_cast<const float4 *>(from + 128 * h);
                    s[h].x = fmaf(v.x, f, s[h].x);
                    s[h].y = fmaf(v.y, f, s[h].y);
                    s[h].z = fmaf(v.z, f, s[h].z);
                    s[h].w = fmaf(v.w, f, s[h].w);
                }
        }
    }
    if (split > 1) {
        sums[warp][lane] = s[0];
        sums[warp][32 + lane] = s[1];
        if (lane == 0) ls[warp] = l;
        __syncthreads();
        if (part != 0) return;
        for (int v = warp + 1; v < warp + split; ++v) {
            l += ls[v];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 x = sums[v][32 * h + lane];
                s[h] = make_float4(s[h].x + x.x, s[h].y + x.y, s[h].z + x.z, s[h].w + x.w);
            }
        }
    }
    if (r >= p.rows) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t row = out_row(a, p, r);
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (4 * lane + 128 * h < D) {
            const float y[4] = {s[h].x * inv, s[h].y * inv, s[h].z * inv, s[h].w * inv};
            store_vec<T, 4>(static_cast<T *>(a.o) + row * D + 4 * lane + 128 * h, y);
        }
    if (lane == 0 && a.lse != nullptr) a.lse[row] = lse_of(m, l);
}

template <typename T>
cudaError_t launch_join(const Args &a, cudaStream_t stream) {
    const int64_t items = (int64_t)a.B * a.per_seq;
    // about as many pieces as an item is cut into when all are of one length
    int split = 1;
    while (split < kJoinWarps && split * 2 * items <= a.workers) split *= 2;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    const int rows = a.T * a.group < a.rows ? a.T * a.group : a.rows;
    cfg.gridDim = dim3((unsigned)items, (unsigned)ceil_div(rows, kJoinWarps / split));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<T>, a, split);
}

int elem_size(int dtype) { return dtype == KDA_DTYPE_BF16 ? 2 : 4; }

int check(const kda_attn_step_params &p) {
    if (p.B < 1 || p.T < 0 || p.q_heads < 1 || !(fabsf(p.scale) < INFINITY)) return KDA_ERR_INVALID_ARG;
    if (p.dtype != KDA_DTYPE_BF16 && p.dtype != KDA_DTYPE_F32) return KDA_ERR_UNSUPPORTED;
    const int st = cache_check(p.cache, p.dtype);
    if (st != KDA_OK) return st;
    if (p.q_heads % p.cache.heads != 0) return KDA_ERR_INVALID_ARG;
    if (p.T != 0 && (p.q == nullptr || p.o == nullptr)) return KDA_ERR_INVALID_ARG;
    const int64_t dense = (int64_t)p.q_heads * p.cache.D;
    if (p.q_stride != 0 && p.q_stride < dense) return KDA_ERR_INVALID_ARG;
    if ((int64_t)p.B * p.T * p.q_heads >= (int64_t)1 << 31 || (int64_t)p.T * (p.q_heads / p.cache.heads) >= (int64_t)1 << 24)
        return KDA_ERR_UNSUPPORTED;
    if (!aligned(p.q, 16) || !aligned(p.o, 16) || !aligned(p.lse, 4) || (p.q_stride * elem_size(p.dtype)) % 16 != 0)
        return KDA_ERR_ALIGNMENT;
    return KDA_OK;
}

Args make(const kda_attn_step_params &p, unsigned int *err) {
    Args a{};
    a.q = p.q;
    a.o = p.o;
    a.lse = p.lse;
    a.q_stride = p.q_stride != 0 ? p.q_stride : (int64_t)p.q_heads * p.cache.D;
    a.B = p.B;
    a.T = p.T;
    a.Hq = p.q_heads;
    a.group = p.q_heads / p.cache.heads;
    a.scale_log2 = p.scale * kLog2e;
    a.cache = cache_args(p.cache, err);
    const int all = a.T * a.group;
    const bool f32 = p.dtype == KDA_DTYPE_F32;
    a.rows = f32 ? fma_rows(all, a.cache.D) : mma_rows(all, a.cache.D);
    a.per_seq = (int)ceil_div(all, a.rows) * a.cache.heads;
    a.unit = f32 ? fma_unit(a) : mma_unit(a);
    a.workers = sm_count() * (f32 ? fma_blocks(a) : mma_blocks(a)) * kWarps;
    return a;
}
size_t bytes_of(const Args &a) { return (size_t)2 * a.workers * a.rows * (a.cache.D + 2) * sizeof(float); }

}  // namespace
}  // namespace attn
}  // namespace kda

extern "C" {

size_t kda_attn_step_workspace(const kda_attn_step_params *p) {
    using namespace kda;
    if (p == nullptr || attn::check(*p) != KDA_OK || p->T == 0) return 0;
    return attn::bytes_of(attn::make(*p, nullptr));
}

int kda_attn_step(const kda_attn_step_params *p, cudaStream_t stream) {
    using namespace kda;
    using namespace kda::attn;
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    const int st = attn::check(*p);
    if (st != KDA_OK || p->T == 0) return st;
    unsigned int *err = nullptr;
    cudaError_t e = device_error_word(&err);
    if (e != cudaSuccess) return status_of_cuda(e);
    Args a = attn::make(*p, err);
    if (a.workers == 0) return status_of_cuda(cudaErrorInvalidDevice);
    if ((int64_t)a.B * a.per_seq >= (int64_t)1 << 31) return KDA_ERR_UNSUPPORTED;
    const size_t bytes = bytes_of(a);
    if (p->workspace != nullptr && p->workspace_bytes < bytes) return KDA_ERR_INVALID_ARG;
    if (!aligned(p->workspace, 16)) return KDA_ERR_ALIGNMENT;
    Scratch ws;
    e = ws.get(p->workspace, bytes, stream);
    if (e != cudaSuccess) return status_of_cuda(e);
    a.pieces = static_cast<float *>(ws.ptr);
    const bool f32 = p->dtype == KDA_DTYPE_F32;
    e = f32 ? launch_attn_fma(a, stream) : launch_attn_mma(a, stream);
    if (e == cudaSuccess) e = f32 ? launch_join<float>(a, stream) : launch_join<bf16>(a, stream);
    return status_of_cuda(ws.release(e));
}

}  // extern "C"
