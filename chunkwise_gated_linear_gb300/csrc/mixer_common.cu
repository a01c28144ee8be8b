// The sum of per-block partial results shared by the token-mixer operators' backward passes.
#include "mixer_common.cuh"

#include <mutex>

namespace kda {
namespace mix {

namespace {

// 32 columns per block; thread (x, y) adds the parts y, y + 32, ... of column x, then the 32
// partial sums are added in the order of y: the result does not depend on timing. Bound by
// reading the partials once (they were just written and mostly lie in L2).
constexpr int kCols = 32, kLanes = 32;

__global__ void __launch_bounds__(kCols *kLanes) sum_partials_kernel(const float *partial, int64_t parts, int64_t total,
                                                                      SumOuts outs) {
    __shared__ float red[kLanes][kCols + 1];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * kCols + x;
    float s = 0.f;
    if (c < total) {
        float s1 = 0.f, s2 = 0.f, s3 = 0.f;
        int64_t p = y;
        for (; p + 3 * kLanes < parts; p += 4 * kLanes) {
            s += partial[p * total + c];
            s1 += partial[(p + kLanes) * total + c];
            s2 += partial[(p + 2 * kLanes) * total + c];
            s3 += partial[(p + 3 * kLanes) * total + c];
        }
        for (; p < parts; p += kLanes) s += partial[p * total + c];
        s = (s + s1) + (s2 + s3);
    }
    red[y][x] = s;
    __syncthreads();
    if (y == 0 && c < total) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < kLanes; ++i) t += red[i][x];
        int64_t at = c;
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
    sum_partials_kernel<<<(unsigned)ceil_div(total, kCols), kCols * kLanes, 0, stream>>>(partial, parts, total, outs);
    return cudaGetLastError();
}

}  // namespace mix
}  // namespace kda
