// Attention over a paged cache (kda_attention.h): the checks and the join of the pieces of items that were cut.
#include "attn_launch.h"

namespace kda {
namespace attn {
namespace {

constexpr int kJoinWarps = 4;

// A warp per query row of an item that was cut: the largest m of its pieces, then sum of 2^(m - max) (l, O) over
// them in the order of the blocks. A block with nothing to join ends after the plan.
template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_join_kernel(const __grid_constant__ Args a) {
    __shared__ int64_t mem[2 * kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x / a.per_seq, item = blockIdx.x - b * a.per_seq;
    const Before n = tiles_before<32 * kJoinWarps>(a, b, mem);
    const int grid = sharers(a.grid, n.total);
    const int len = cache_len(a.cache, b), tiles = tiles_of(len);
    const int64_t begin = n.upto + (int64_t)item * tiles;
    const int w0 = owner(n.total, begin, grid), w1 = owner(n.total, begin + tiles - 1, grid);
    if (w0 == w1) return;
    const Piece p = piece_at(a, b, len, (int64_t)item * tiles, tiles);
    const int D = a.cache.D, r = blockIdx.y * kJoinWarps + warp;
    if (r >= p.rows) return;
    const int64_t size = (int64_t)a.rows * (D + 2);
    // the piece of the first block begins there (slot 1), the others come from the block before (slot 0)
    auto piece = [&](int w) { return a.pieces + (int64_t)(2 * w + (w == w0 ? 1 : 0)) * size; };
    float m = -INFINITY;
    for (int w = w0 + lane; w <= w1; w += 32) m = fmaxf(m, piece(w)[(int64_t)a.rows * D + 2 * r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, s[8] = {};
#pragma unroll 4
    for (int w = w0; w <= w1; ++w) {
        const float *from = piece(w);
        const float2 x = *reinterpret_cast<const float2 *>(from + (int64_t)a.rows * D + 2 * r);
        const float f = tc5::ex2(x.x - ref);
        l = fmaf(x.y, f, l);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (lane + 32 * j < D) s[j] = fmaf(from[(int64_t)r * D + lane + 32 * j], f, s[j]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t row = out_row(a, p, r);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (lane + 32 * j < D) static_cast<T *>(a.o)[row * D + lane + 32 * j] = from_f<T>(s[j] * inv);
    if (lane == 0 && a.lse != nullptr) a.lse[row] = lse_of(m, l);
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
    a.rows = f32 ? fma_rows(all) : mma_rows(all, a.cache.D);
    a.row_blocks = (int)ceil_div(all, a.rows);
    a.per_seq = a.row_blocks * a.cache.heads;
    a.grid = sm_count() * (f32 ? fma_blocks(a) : mma_blocks(a));
    return a;
}
size_t bytes_of(const Args &a) { return (size_t)2 * a.grid * a.rows * (a.cache.D + 2) * sizeof(float); }

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
    if (a.grid == 0) return status_of_cuda(cudaErrorInvalidDevice);
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
    if (e == cudaSuccess) {
        const dim3 grid((unsigned)(a.B * a.per_seq), (unsigned)ceil_div(a.rows, kJoinWarps));
        if (f32)
            attn_join_kernel<float><<<grid, 32 * kJoinWarps, 0, stream>>>(a);
        else
            attn_join_kernel<bf16><<<grid, 32 * kJoinWarps, 0, stream>>>(a);
        e = cudaGetLastError();
    }
    return status_of_cuda(ws.release(e));
}

}  // extern "C"
