// The sum of per-block partial results shared by the token-mixer operators' backward passes.
#include "mixer_common.cuh"

#include <mutex>

namespace kda {
namespace mix {

namespace {

// A block takes 32 V columns: thread (x, y) adds the parts y, y + LANES, ... of columns V x .. V x + V - 1, then the
// LANES sums are added in the order of y: the result does not depend on timing. Bound by
// reading the partials once (they were just written and mostly lie in L2). Few columns: one each and 32 lanes, for
// enough blocks; many: four at a time and 8 lanes (50 parts of 61440 columns: 17 -> 5 us).
template <int V, int LANES>
__global__ void __launch_bounds__(32 * LANES) sum_partials_kernel(const float *partial, int64_t parts, int64_t total, SumOuts outs) {
    __shared__ float red[LANES][32 * V + 1];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t c = ((int64_t)blockIdx.x * 32 + x) * V;
    float s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = 0.f;
    if (c < total) {
        const float *p = partial + c;
        constexpr int kAhead = 4;
        for (int64_t q = y; q < parts; q += kAhead * LANES) {
            float t[kAhead][V];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (q + k * LANES < parts) load_vec<float, V>(t[k], p + (q + k * LANES) * total);
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (q + k * LANES < parts)
#pragma unroll
                    for (int v = 0; v < V; ++v) s[v] += t[k][v];
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) red[y][x * V + v] = s[v];
    __syncthreads();
    for (int e = threadIdx.x; e < 32 * V; e += 32 * LANES) {
        int64_t at = (int64_t)blockIdx.x * 32 * V + e;
        if (at >= total) break;
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < LANES; ++i) t += red[i][e];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (at >= 0 && at < outs.len[k] && outs.out[k] != nullptr) outs.out[k][at] = t;
            at -= outs.len[k];
        }
    }
}

std::once_flag g_sm_once[64];
int g_sm[64];

}  // namespace

int sm_count() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::call_once(g_sm_once[dev], [dev] {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) g_sm[dev] = n;
    });
    return g_sm[dev];
}

cudaError_t launch_sum_partials(const float *partial, int64_t parts, int64_t total, const SumOuts &outs, cudaStream_t stream) {
    if (total == 0) return cudaSuccess;
    if (total % 4 == 0 && total >= 16384 && aligned(partial, 16))
        sum_partials_kernel<4, 8><<<(unsigned)ceil_div(total, 128), 256, 0, stream>>>(partial, parts, total, outs);
    else
        sum_partials_kernel<1, 32><<<(unsigned)ceil_div(total, 32), 1024, 0, stream>>>(partial, parts, total, outs);
    return cudaGetLastError();
}

}  // namespace mix
}  // namespace kda
