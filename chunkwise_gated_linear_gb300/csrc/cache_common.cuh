// The paged key-value cache of kda_attention.h on the device: where a token lies, and rows of 8-bit
// values with one power of two each.
#pragma once

#include <cuda_fp16.h>

#include "kda_attention.h"
#include "mixer_common.cuh"

namespace kda {

constexpr unsigned int kDeviceErrCache = 4u;  // KDA_DEVICE_ERR_CACHE

namespace mix {

// Lengths and pages are read from device memory and may hold anything: each is checked where it is read.
struct Cache {
    void *k, *v;
    uint8_t *ks, *vs;  // null: values in the type of the data
    int64_t page_rows;     // rows (of D elements) between pages
    int64_t scale_stride;  // bytes between pages of the scales
    const int32_t *table;
    int64_t table_stride;
    const int32_t *lens;
    int pages, heads, page, D, max_pages;
    int shift;       // page == 1 << shift, or -1
    int most;        // max_pages * page, at most 2^31 - 65 (sums with a few more stay in range)
    unsigned int *err;
};

// The length of sequence b, within what the table can hold.
__device__ __forceinline__ int cache_len(const Cache &c, int b) {
    const int n = c.lens[b];
    const int m = n < 0 ? 0 : (n > c.most ? c.most : n);
    if (m != n) atomicOr(c.err, kDeviceErrCache);
    return m;
}
// Page and row within it of position pos >= 0.
__device__ __forceinline__ void cache_split(const Cache &c, int pos, int &page, int &slot) {
    if (c.shift >= 0) {
        page = pos >> c.shift;
        slot = pos & (c.page - 1);
    } else {
        page = pos / c.page;
        slot = pos - page * c.page;
    }
}
// The page of sequence b that holds position pos of it (0 <= pos < c.most) and the row within that; -1 and the error
// bit where the table names no page of the cache.
__device__ __forceinline__ int cache_page(const Cache &c, int b, int pos, int &slot) {
    int at;
    cache_split(c, pos, at, slot);
    const int page = c.table[(int64_t)b * c.table_stride + at];
    if ((unsigned)page < (unsigned)c.pages) return page;
    atomicOr(c.err, kDeviceErrCache);
    return -1;
}
// Offsets in rows (of D elements) and in scale bytes.
__device__ __forceinline__ int64_t cache_row(const Cache &c, int page, int head, int slot) {
    return (int64_t)page * c.page_rows + (int64_t)head * c.page + slot;
}
__device__ __forceinline__ int64_t cache_scale(const Cache &c, int page, int head, int slot) {
    return (int64_t)page * c.scale_stride + (int64_t)head * c.page + slot;
}

// ---- rows of 8-bit values ------------------------------------------------------------------
// The exponent of a row whose largest finite |x| is `top`: the least e >= -126 with top <= 448 2^e = 1.75 2^(8 + e). With
// top = f 2^x, e = x - 8, and one more where f > 1.75: adding 2^21 - 1 to the bits carries into the exponent just then.
__device__ __forceinline__ int row_exponent(float top) {
    const int e = (int)((__float_as_uint(top) + 0x1fffffu) >> 23) - 135;
    return e < -126 ? -126 : e;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 <= e <= 127
// |x|, or 0 where x is not finite
__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a < INFINITY ? a : 0.f;
}
// Two floats to e4m3, `lo` in the low byte: nearest even; infinities become 448, NaN stays.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    unsigned short d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ void e4m3_to_f(uint32_t pair, float &lo, float &hi) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)pair));
    const __half2 v = *reinterpret_cast<__half2 *>(&h);
    lo = __low2float(v);
    hi = __high2float(v);
}

// ---- host side -----------------------------------------------------------------------------
// Checks of a cache against the data type of a call.
inline int cache_check(const kda_kv_cache &c, int dtype) {
    if (c.k == nullptr || c.v == nullptr || c.block_table == nullptr || c.lens == nullptr) return KDA_ERR_INVALID_ARG;
    if (c.pages < 1 || c.heads < 1 || c.page_size < 1 || c.max_pages < 1 || c.D < 1) return KDA_ERR_INVALID_ARG;
    if (c.dtype != KDA_DTYPE_E4M3 && c.dtype != dtype) return KDA_ERR_UNSUPPORTED;
    if (c.D % 16 != 0 || c.D > 256) return KDA_ERR_UNSUPPORTED;
    const bool e4m3 = c.dtype == KDA_DTYPE_E4M3;
    if (e4m3 != (c.k_scale != nullptr) || e4m3 != (c.v_scale != nullptr)) return KDA_ERR_INVALID_ARG;
    const int64_t dense = (int64_t)c.heads * c.page_size;
    if (dense > ((int64_t)1 << 31) / c.pages) return KDA_ERR_UNSUPPORTED;  // so that its products below stay in 64 bits
    const int64_t stride = c.page_stride == 0 ? dense * c.D : c.page_stride;
    if (stride < dense * c.D || stride % c.D != 0) return KDA_ERR_INVALID_ARG;
    if (c.scale_stride != 0 && c.scale_stride < dense) return KDA_ERR_INVALID_ARG;
    if (c.table_stride != 0 && c.table_stride < c.max_pages) return KDA_ERR_INVALID_ARG;
    if (stride / c.D > ((int64_t)1 << 31) / c.pages) return KDA_ERR_UNSUPPORTED;
    if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.block_table, 4) || !aligned(c.lens, 4)) return KDA_ERR_ALIGNMENT;
    return KDA_OK;
}
inline Cache cache_args(const kda_kv_cache &c, unsigned int *err) {
    Cache a{};
    a.k = c.k;
    a.v = c.v;
    a.ks = c.k_scale;
    a.vs = c.v_scale;
    const int64_t dense = (int64_t)c.heads * c.page_size;
    a.page_rows = c.page_stride == 0 ? dense : c.page_stride / c.D;
    a.scale_stride = c.scale_stride == 0 ? dense : c.scale_stride;
    a.table = c.block_table;
    a.table_stride = c.table_stride == 0 ? c.max_pages : c.table_stride;
    a.lens = c.lens;
    a.pages = c.pages;
    a.heads = c.heads;
    a.page = c.page_size;
    a.D = c.D;
    a.max_pages = c.max_pages;
    a.shift = -1;
    for (int s = 0; s < 31; ++s)
        if (c.page_size == 1 << s) a.shift = s;
    const int64_t most = (int64_t)c.max_pages * c.page_size;
    a.most = (int)(most > INT32_MAX - 64 ? INT32_MAX - 64 : most);
    a.err = err;
    return a;
}

}  // namespace mix
}  // namespace kda
