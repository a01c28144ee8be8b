// Attention over a paged cache (kda_attention.h): the checks and the join of the pieces of items that were cut.
#include "attn_launch.h"

namespace kda {
namespace attn {
namespace {

constexpr int kSplit = 16;  // warps for a row, at most
constexpr int join_warps(int lc) { return lc == 8 ? kSplit : 8; }  // of a block, at most

// A query row of an item that was cut: with the largest m of its pieces, the sum of 2^(m - max) (l, O) over them. `split` warps
// share a row's pieces in order, each with a maximum of its own, and are then added up. Of a warp, LC lanes hold four
// channels each and the others take other pieces: 32 for many rows, 8 (and a block for every 32 channels) for few. The
// workers of the attention have left word where the pieces of an item begin and end. What it costs is waiting, for the
// attention's end, for that word and for the pieces, of which a warp reads all statistics and the first few at once: 4 to 6
// us behind the attention. It is launched early, which saves 1 to 4 of them. (One sequence of 131071 tokens, 228 pieces a
// row, both kernels: 102 us with 8 warps for a row, 96 with 16, 94 with a block for every 32 channels; 91 since the ends
// are told, as a plan of its own, with the registers that the attention takes, did not run before its end.)
template <typename T, int LC>
__global__ void __launch_bounds__(32 * join_warps(LC), 2) attn_join_kernel(const __grid_constant__ Args a, int split) {
    constexpr int kAtOnce = 32 / LC, kPasses = LC == 8 ? 1 : 2;  // pieces of a warp at a time; turns over its channels
    constexpr int kAhead = LC == 8 ? 4 : 2;  // pieces read before the statistics are here
    __shared__ float4 sums[join_warps(LC)][kPasses * LC];
    __shared__ float2 stat[join_warps(LC)];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    Piece p;  // the item
    p.b = blockIdx.x / a.per_seq;
    const int item = blockIdx.x - p.b * a.per_seq, rb = item / a.cache.heads;
    p.head = item - rb * a.cache.heads;
    p.row0 = rb * a.rows;
    p.rows = a.T * a.group - p.row0 < a.rows ? a.T * a.group - p.row0 : a.rows;
    wait_for_previous();
    const int w0 = a.ends[blockIdx.x].x, w1 = a.ends[blockIdx.x].y;
    if (w0 == w1) return;
    const int D = a.cache.D, part = warp % split;
    const int r = blockIdx.y * (warps / split) + warp / split;
    const int each = (w1 - w0 + split) / split;  // pieces of a warp
    const int from = w0 + part * each, to = from + each < w1 + 1 ? from + each : w1 + 1;
    float m = -INFINITY, l = 0.f;
    float4 s[kPasses];
#pragma unroll
    for (int h = 0; h < kPasses; ++h) s[h] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int mine_of = lane / LC, d0 = (LC == 8 ? 32 * (int)blockIdx.z : 0) + 4 * (lane % LC);
    auto scale = [&](float f) {
        l *= f;
#pragma unroll
        for (int h = 0; h < kPasses; ++h) s[h] = make_float4(s[h].x * f, s[h].y * f, s[h].z * f, s[h].w * f);
    };
    if (r < p.rows) {
        // pieces 2 w, and of the first worker, where the item begins, 2 w + 1
        const int64_t size = (int64_t)a.rows * (D + 2);
#pragma unroll 1
        for (int w = from; w < to; w += 32) {
            const int my = w + lane < to ? w + lane : w, count = to - w < 32 ? to - w : 32;
            const float2 x = reinterpret_cast<const float2 *>(a.pieces + (2 * my + (my == w0)) * size + (int64_t)a.rows * D)[r];
            const float *o = a.pieces + 2 * w * size + (int64_t)r * D + d0;
            auto load = [&](int i, int h) {
                return i < count && d0 + 128 * h < D ? *reinterpret_cast<const float4 *>(o + (2 * i + (w + i == w0)) * size + 128 * h)
                                                     : make_float4(0.f, 0.f, 0.f, 0.f);
            };
            float4 first[kAhead][kPasses];
#pragma unroll
            for (int t = 0; t < kAhead; ++t)
#pragma unroll
                for (int h = 0; h < kPasses; ++h) first[t][h] = load(mine_of + t * kAtOnce, h);
            float top = x.x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (top > m) {
                scale(tc5::ex2(m - top));
                m = top;
            }
            float f = tc5::ex2(x.x - (m == -INFINITY ? 0.f : m));
            float ls = w + lane < to ? x.y * f : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
            l += ls;
            auto add = [&](int i, int h, const float4 &v) {
                const float fi = __shfl_sync(0xffffffffu, f, i & 31);
                if (i < count) s[h] = make_float4(fmaf(v.x, fi, s[h].x), fmaf(v.y, fi, s[h].y), fmaf(v.z, fi, s[h].z), fmaf(v.w, fi, s[h].w));
            };
#pragma unroll
            for (int t = 0; t < kAhead; ++t)
#pragma unroll
                for (int h = 0; h < kPasses; ++h) add(mine_of + t * kAtOnce, h, first[t][h]);
#pragma unroll 2
            for (int i = mine_of + kAhead * kAtOnce; i - mine_of < count; i += kAtOnce)
#pragma unroll
                for (int h = 0; h < kPasses; ++h) add(i, h, load(i, h));
        }
        if constexpr (LC < 32) {
#pragma unroll
            for (int off = LC; off < 32; off <<= 1) {
                s[0].x += __shfl_xor_sync(0xffffffffu, s[0].x, off);
                s[0].y += __shfl_xor_sync(0xffffffffu, s[0].y, off);
                s[0].z += __shfl_xor_sync(0xffffffffu, s[0].z, off);
                s[0].w += __shfl_xor_sync(0xffffffffu, s[0].w, off);
            }
        }
    }
    if (split > 1) {
        if (lane < LC) {
#pragma unroll
            for (int h = 0; h < kPasses; ++h) sums[warp][h * LC + lane] = s[h];
        }
        if (lane == 0) stat[warp] = make_float2(m, l);
        __syncthreads();
        if (part != 0) return;
#pragma unroll 1
        for (int v = warp + 1; v < warp + split; ++v) {
            const float2 x = stat[v];
            if (x.x > m) {
                scale(tc5::ex2(m - x.x));
                m = x.x;
            }
            const float f = tc5::ex2(x.x - (m == -INFINITY ? 0.f : m));
            l = fmaf(x.y, f, l);
#pragma unroll
            for (int h = 0; h < kPasses; ++h) {
                const float4 y = sums[v][h * LC + lane % LC];
                s[h] = make_float4(fmaf(y.x, f, s[h].x), fmaf(y.y, f, s[h].y), fmaf(y.z, f, s[h].z), fmaf(y.w, f, s[h].w));
            }
        }
    }
    if (r >= p.rows || lane >= LC) return;
    const bool empty = l == 0.f;  // zeros, whatever the values are
    const float inv = 1.f / l;
    const int64_t row = out_row(a, p, r);
#pragma unroll
    for (int h = 0; h < kPasses; ++h)
        if (d0 + 128 * h < D) {
            const float y[4] = {empty ? 0.f : s[h].x * inv, empty ? 0.f : s[h].y * inv, empty ? 0.f : s[h].z * inv, empty ? 0.f : s[h].w * inv};
            store_vec<T, 4>(static_cast<T *>(a.o) + row * D + d0 + 128 * h, y);
        }
    if (d0 == 0 && a.lse != nullptr) a.lse[row] = lse_of(m, l);
}

int64_t items_of(const Args &a) { return (int64_t)a.B * a.per_seq; }

template <typename T>
cudaError_t launch_join(const Args &a, cudaStream_t stream) {
    const int64_t items = items_of(a);
    const int rows = a.T * a.group < a.rows ? a.T * a.group : a.rows;
    // Warps for a row: so many that about 16 on every SM have something to do, but not below four pieces each when all items are of one
    // length. (Blocks of 8 warps instead of 16 where rows share them: 8 sequences of up to 700 tokens 13.3 -> 12.6 us, wide
    // heads 58 -> 57 us.)
    int split = 1;
    while (split < kSplit && split * 8 * items <= a.workers && split * items * rows < 16 * (int64_t)sm_count()) split *= 2;
    const bool few = split == kSplit;
    const int most = join_warps(few ? 8 : 32) / split, at_once = most < rows ? most : rows;  // rows of a block
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)items, (unsigned)ceil_div(rows, at_once), few ? (unsigned)ceil_div(a.cache.D, 32) : 1u);
    cfg.blockDim = dim3((unsigned)(32 * split * at_once));
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return few ? cudaLaunchKernelEx(&cfg, attn_join_kernel<T, 8>, a, split) : cudaLaunchKernelEx(&cfg, attn_join_kernel<T, 32>, a, split);
}

int elem_size(int dtype) { return dtype == KDA_DTYPE_BF16 ? 2 : 4; }

int check(const kda_attn_step_params &p) {
    if (p.B < 1 || p.T < 0 || p.q_heads < 1 || !(fabsf(p.scale) < INFINITY)) return KDA_ERR_INVALID_ARG;
    if (p.dtype != KDA_DTYPE_BF16 && p.dtype != KDA_DTYPE_F32) return KDA_ERR_UNSUPPORTED;
    const int st = cache_check(p.cache, p.dtype);
    if (st != KDA_OK) return st;
    if (p.q_heads % p.cache.heads != 0) return KDA_ERR_INVALID_ARG;
    if (p.q_heads / p.cache.heads > 256) return KDA_ERR_UNSUPPORTED;
    if (p.T != 0 && (p.q == nullptr || p.o == nullptr)) return KDA_ERR_INVALID_ARG;
    const int64_t dense = (int64_t)p.q_heads * p.cache.D;
    if (p.q_stride != 0 && p.q_stride < dense) return KDA_ERR_INVALID_ARG;
    if ((int64_t)p.B * p.T * p.q_heads >= (int64_t)1 << 31 || (int64_t)p.T * (p.q_heads / p.cache.heads) >= (int64_t)1 << 24)
        return KDA_ERR_UNSUPPORTED;
    if (!aligned(p.q, 16) || !aligned(p.o, 16) || !aligned(p.lse, 4) || (p.q_stride * elem_size(p.dtype)) % 16 != 0)
        return KDA_ERR_ALIGNMENT;
    return KDA_OK;
}

Args make(const kda_attn_step_params &p) {
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
    a.cache = cache_args(p.cache, nullptr);
    const int all = a.T * a.group;
    const bool f32 = p.dtype == KDA_DTYPE_F32;
    a.rows = f32 ? fma_rows(all) : mma_rows(all, a.cache.D);
    a.group_magic = (uint32_t)ceil_div((int64_t)1 << 32, a.group);  // not used for 1
    a.row_blocks = (int)ceil_div(all, a.rows);
    a.per_seq = a.row_blocks * a.cache.heads;
    a.unit_shift = f32 ? fma_unit_shift(a) : mma_unit_shift(a);
    a.workers = sm_count() * (f32 ? fma_workers(a) : mma_workers(a));
    return a;
}
// Whether the units and costs of all items, were all sequences as long as the table allows, are counted in 32 bits.
bool in_range(const Args &a) {
    const int64_t weight = ((int64_t)a.cache.most >> a.unit_shift) + 1 + kItemCost;
    return items_of(a) <= (int64_t)UINT32_MAX / weight;
}
size_t pieces_of(const Args &a) { return (size_t)2 * a.workers * a.rows * (a.cache.D + 2); }
size_t bytes_of(const Args &a) { return pieces_of(a) * sizeof(float) + (size_t)items_of(a) * sizeof(int2); }

}  // namespace
}  // namespace attn
}  // namespace kda

extern "C" {

size_t kda_attn_step_workspace(const kda_attn_step_params *p) {
    using namespace kda;
    if (p == nullptr || attn::check(*p) != KDA_OK || p->T == 0) return 0;
    const attn::Args a = attn::make(*p);
    return attn::in_range(a) ? attn::bytes_of(a) : 0;
}

int kda_attn_step(const kda_attn_step_params *p, cudaStream_t stream) {
    using namespace kda;
    using namespace kda::attn;
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    const int st = attn::check(*p);
    if (st != KDA_OK || p->T == 0) return st;
    Args a = attn::make(*p);
    if (!in_range(a)) return KDA_ERR_UNSUPPORTED;
    cudaError_t e = device_error_word(&a.cache.err);
    if (e != cudaSuccess) return status_of_cuda(e);
    if (a.workers == 0) return status_of_cuda(cudaErrorInvalidDevice);
    const size_t bytes = bytes_of(a);
    if (p->workspace != nullptr && p->workspace_bytes < bytes) return KDA_ERR_INVALID_ARG;
    if (!aligned(p->workspace, 16)) return KDA_ERR_ALIGNMENT;
    Scratch ws;
    e = ws.get(p->workspace, bytes, stream);
    if (e != cudaSuccess) return status_of_cuda(e);
    a.pieces = static_cast<float *>(ws.ptr);
    a.ends = reinterpret_cast<int2 *>(a.pieces + pieces_of(a));
    const bool f32 = p->dtype == KDA_DTYPE_F32;
    e = f32 ? launch_attn_fma(a, stream) : launch_attn_mma(a, stream);
    if (e == cudaSuccess) e = f32 ? launch_join<float>(a, stream) : launch_join<bf16>(a, stream);
    return status_of_cuda(ws.release(e));
}

}  // extern "C"
