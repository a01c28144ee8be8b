// The end of a piece, the join of pieces, and launching, for the kernels of attention over a paged cache.
#pragma once

#include <atomic>

#include "attn_common.cuh"

namespace kda {
namespace attn {

// Query rows of an item for `all` rows of a sequence and key head, blocks on an SM, and the launch, of the kernel for
// fp32 data and of that for bf16.
int fma_rows(int all);
int fma_blocks(const Args &a);
cudaError_t launch_attn_fma(const Args &a, cudaStream_t stream);
int mma_rows(int all, int D);
int mma_blocks(const Args &a);
cudaError_t launch_attn_mma(const Args &a, cudaStream_t stream);

// The warps' results of a piece, O [rows][PITCH] at `mem` + warp * `stride` bytes and (m, l) in ml [warp][RB], put together: into
// o and lse where the piece is a whole item, otherwise into the block's piece of scratch.
template <typename T, int DP, int RB, int PITCH>
__device__ __forceinline__ void finish(const Args &a, const Piece &p, const unsigned char *mem, int stride, const float2 *ml, int block) {
    const bool whole = p.t0 == 0 && p.t1 == p.tiles;
    const int D = a.cache.D;
    float *piece = a.pieces + (int64_t)(2 * block + (p.t0 == 0 ? 1 : 0)) * a.rows * (D + 2);
    for (int i = threadIdx.x; i < p.rows * (DP / 4); i += kThreads) {
        const int r = i / (DP / 4), d = (i - r * (DP / 4)) * 4;
        if (d >= D) continue;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, ml[w * RB + r].x);
        const float ref = m == -INFINITY ? 0.f : m;
        float l = 0.f;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float2 x = ml[w * RB + r];
            const float f = tc5::ex2(x.x - ref);
            const float4 v = *reinterpret_cast<const float4 *>(mem + w * stride + (r * PITCH + d) * 4);
            l = fmaf(x.y, f, l);
            s.x = fmaf(v.x, f, s.x);
            s.y = fmaf(v.y, f, s.y);
            s.z = fmaf(v.z, f, s.z);
            s.w = fmaf(v.w, f, s.w);
        }
        if (whole) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int64_t row = out_row(a, p, r);
            const float y[4] = {s.x * inv, s.y * inv, s.z * inv, s.w * inv};
            store_vec<T, 4>(static_cast<T *>(a.o) + row * D + d, y);
            if (d == 0 && a.lse != nullptr) a.lse[row] = lse_of(m, l);
        } else {
            float *to = piece + (int64_t)r * D + d;
            *reinterpret_cast<float2 *>(to) = make_float2(s.x, s.y);
            *reinterpret_cast<float2 *>(to + 2) = make_float2(s.z, s.w);
            if (d == 0) *reinterpret_cast<float2 *>(piece + (int64_t)a.rows * D + 2 * r) = make_float2(m, l);
        }
    }
}

// Launches a kernel of kSmem bytes of shared memory, as many blocks as there are (a.grid).
template <auto kernel, int kSmem>
cudaError_t launch_kernel(const Args &a, cudaStream_t stream) {
    static std::atomic<bool> ready[64];  // per device, of this kernel
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_release);
    }
    kernel<<<a.grid, kThreads, kSmem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace attn
}  // namespace kda
