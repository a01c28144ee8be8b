// Attention over a paged cache (kda_attention.h), what its kernels share: how the work is cut, how keys and values
// stream in, and how the pieces of one result are joined.
//
// An item is one (sequence, block of query rows, key head); its keys are cut into tiles of 64. All items' tiles, one after
// another, are dealt out in equal shares to the blocks of the grid, so that a block has at most one item that began in
// the block before and one that goes on in the next. Such pieces leave (m, l, O) in scratch: the reference m of their
// exponentials 2^(s - m), the sum l of those, and O = sum 2^(s - m) v; a second kernel joins them in the order of
// the blocks. Which items are cut follows from the lengths and sizes alone, so results repeat bit for bit.
//
// Query rows of an item are the (token, head of the group) pairs t * group + g of one key head, in blocks of
// `rows`; the keys that row sees are those at positions below len - T + t + 1.
#pragma once

#include "cache_common.cuh"

namespace kda {
namespace attn {

using namespace mix;

constexpr int kTile = 64;              // keys of a tile
constexpr int kWarps = 4;              // of a block
constexpr int kThreads = 32 * kWarps;

struct Args {
    const void *q;
    void *o;
    float *lse;
    int64_t q_stride;
    int B, T, Hq, group;
    int rows;        // query rows of an item (at most)
    int row_blocks;  // ceil(T * group / rows)
    int per_seq;     // items of a sequence: row_blocks * heads
    float scale_log2;  // scale * log2 e
    Cache cache;
    float *pieces;   // [2 grid][rows][D + 2]: O, then m and l
    int grid;
};

__device__ __forceinline__ int tiles_of(int len) { return len <= kTile ? 1 : (len + kTile - 1) / kTile; }

// The first tile of block w's share of `total`, and the block that has tile x in its share.
__device__ __forceinline__ int64_t share(int64_t total, int w, int grid) { return total * w / grid; }
__device__ __forceinline__ int owner(int64_t total, int64_t x, int grid) { return (int)(((x + 1) * grid - 1) / total); }

// Number of tiles of all items before sequence `upto`, and of all.
struct Before {
    int64_t upto, total;
};
// Called by all `NT` threads of a block; `mem`: 2 * NT / 32 int64.
template <int NT>
__device__ __forceinline__ Before tiles_before(const Args &a, int upto, int64_t *mem) {
    int64_t lo = 0, all = 0;
    for (int b = threadIdx.x; b < a.B; b += NT) {
        const int n = tiles_of(cache_len(a.cache, b));
        all += n;
        if (b < upto) lo += n;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        lo += __shfl_xor_sync(0xffffffffu, lo, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    if ((threadIdx.x & 31) == 0) {
        mem[2 * (threadIdx.x >> 5)] = lo;
        mem[2 * (threadIdx.x >> 5) + 1] = all;
    }
    __syncthreads();
    lo = all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        lo += mem[2 * w];
        all += mem[2 * w + 1];
    }
    return Before{lo * a.per_seq, all * a.per_seq};
}

// Where a block's share begins: the sequence, the tiles of all items before it, and how many blocks have a share (each
// then has a tile at least).
struct Start {
    int b, grid;
    int64_t before, total;
};
__device__ __forceinline__ int sharers(int grid, int64_t total) { return total < grid ? (int)total : grid; }
// Thread i adds up the sequences i * each .. i * each + each - 1; a scan over the threads finds whose part holds the share's
// first tile. `mem`: kWarps + 2 int64; block w < sharers().
__device__ __forceinline__ Start find_start(const Args &a, int w, int64_t *mem) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int each = (a.B + kThreads - 1) / kThreads;
    const int first = threadIdx.x * each;
    int64_t sum = 0;
    for (int b = first; b < first + each && b < a.B; ++b) sum += tiles_of(cache_len(a.cache, b));
    int64_t scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += x;
    }
    if (lane == 31) mem[warp] = scan;
    __syncthreads();
    int64_t base = 0, total = 0;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) {
        if (v < warp) base += mem[v];
        total += mem[v];
    }
    total *= a.per_seq;
    const int grid = sharers(a.grid, total);
    const int64_t at = share(total, w, grid);
    int64_t before = (base + scan - sum) * a.per_seq;
    if (at >= before && at < before + sum * a.per_seq) {  // one thread's
        int b = first;
        for (;;) {
            const int64_t n = (int64_t)tiles_of(cache_len(a.cache, b)) * a.per_seq;
            if (at < before + n) break;
            before += n;
            ++b;
        }
        mem[kWarps] = b;
        mem[kWarps + 1] = before;
    }
    __syncthreads();
    return Start{(int)mem[kWarps], grid, mem[kWarps + 1], total};
}

// One piece of work: tiles t0 .. t1 - 1 of an item.
struct Piece {
    int b, len, head, row0, rows;  // first query row of the item and how many it has
    int t0, t1, tiles;
    int last;  // keys that the last of its rows sees: no key at or after this one counts
};
__device__ __forceinline__ int seen(const Args &a, int len, int row) {
    const int n = len - a.T + row / a.group + 1;
    return n < 0 ? 0 : n;
}
__device__ __forceinline__ Piece piece_at(const Args &a, int b, int len, int64_t off, int64_t left) {
    Piece p;
    p.b = b;
    p.len = len;
    p.tiles = tiles_of(len);
    const int item = (int)(off / p.tiles);
    p.t0 = (int)(off - (int64_t)item * p.tiles);
    p.t1 = left < p.tiles - p.t0 ? p.t0 + (int)left : p.tiles;
    const int rb = item / a.cache.heads;
    p.head = item - rb * a.cache.heads;
    p.row0 = rb * a.rows;
    const int all = a.T * a.group;
    p.rows = all - p.row0 < a.rows ? all - p.row0 : a.rows;
    p.last = seen(a, len, p.row0 + p.rows - 1);
    return p;
}

// Offsets (elements) of a query row in q, and of its row in o and lse.
__device__ __forceinline__ int64_t q_at(const Args &a, const Piece &p, int r) {
    const int row = p.row0 + r, t = row / a.group;
    return ((int64_t)p.b * a.T + t) * a.q_stride + (int64_t)(p.head * a.group + row - t * a.group) * a.cache.D;
}
__device__ __forceinline__ int64_t out_row(const Args &a, const Piece &p, int r) {
    const int row = p.row0 + r, t = row / a.group;
    return ((int64_t)p.b * a.T + t) * a.Hq + p.head * a.group + row - t * a.group;
}

constexpr float kLn2 = 0.6931471805599453f;
// log of a row's sum of e^score from the reference m (base 2) and the sum l
__device__ __forceinline__ float lse_of(float m, float l) { return l > 0.f ? (m + log2f(l)) * kLn2 : (l == 0.f ? -INFINITY : l); }

// 16 bytes of a row of the cache into shared memory, zeros where `ok` is false.
__device__ __forceinline__ void copy16(uint32_t to, const void *from, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(to), "l"(from), "r"(ok ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// The stream of one warp's keys and values: its KEYS of each step of kWarps * KEYS positions of a piece, through a ring of
// STAGES slots of shared memory that is its own, so that no other warp is waited for. A slot holds KEYS rows of K and of
// V, kPitch bytes each, 16-byte chunk c of row r at chunk c ^ (r & 7): 8 rows at one chunk lie in different
// banks. Rows that no query of the piece sees, or without a page, are zeros.
// The page of a row is read from the table two steps before its copies are issued, and the rows' exponent bytes one step
// before, so that neither is waited for.
template <typename C, int DP, int KEYS, int STAGES>
struct Stream {
    static constexpr int kPitch = DP * (int)sizeof(C) < 128 ? 128 : DP * (int)sizeof(C);
    static constexpr int kHalf = KEYS * kPitch;  // K or V of a slot
    static constexpr int kBytes = STAGES * 2 * kHalf;
    static constexpr int kScaleBytes = STAGES * 2 * KEYS;
    static constexpr int kStep = kWarps * KEYS;
    static constexpr int kChunks = kPitch / 16;            // of a row
    static constexpr int kTurns = KEYS * kChunks / 32;     // copies of a lane for KEYS rows
    static constexpr bool kScaled = sizeof(C) == 1;

    const Args &a;
    uint32_t ring;        // shared address
    uint8_t *scales;      // [STAGES][2][KEYS] exponent bytes
    int lane, warp;
    Piece p;
    int end;              // steps of the piece end here
    int entry, row;       // of this lane's row (lane % KEYS): the table's entry for the step after next, the row of the
    uint32_t sk, sv;      // cache (-1: zeros) and its exponent bytes for the next

    __device__ __forceinline__ Stream(const Args &a_, unsigned char *mem, uint8_t *sc, int lane_, int warp_)
        : a(a_), ring(smem_u32(mem)), scales(sc), lane(lane_), warp(warp_) {}

    __device__ __forceinline__ int position(int s) const { return s * kStep + warp * KEYS + (lane & (KEYS - 1)); }
    __device__ __forceinline__ void look(int s) {
        const int pos = position(s);
        entry = -1;
        if (s < end && pos < p.last) {
            int at, slot;
            cache_split(a.cache, pos, at, slot);
            entry = a.cache.table[(int64_t)p.b * a.cache.table_stride + at];
        }
    }
    __device__ __forceinline__ void resolve(int s) {
        const int pos = position(s);
        row = -1;
        if (s < end && pos < p.last) {
            if ((unsigned)entry < (unsigned)a.cache.pages) {
                int at, slot;
                cache_split(a.cache, pos, at, slot);
                row = (int)cache_row(a.cache, entry, p.head, slot);
                if constexpr (kScaled) {
                    const int64_t x = cache_scale(a.cache, entry, p.head, slot);
                    sk = a.cache.ks[x];
                    sv = a.cache.vs[x];
                }
            } else {
                atomicOr(a.cache.err, kDeviceErrCache);
            }
        }
    }
    // Steps s0 .. s1 - 1 of the piece: the first STAGES - 1 are on their way after this.
    __device__ __forceinline__ void begin(const Piece &piece, int s0, int s1) {
        p = piece;
        end = s1;
        sk = sv = 0;
        look(s0);
        resolve(s0);
        look(s0 + 1);
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) fetch(s0 + i, i);
    }
    __device__ __forceinline__ void fetch(int s, int slot) {
        if (s < end) {
            const int cpr = a.cache.D * (int)sizeof(C) / 16;
            const uint32_t to = ring + slot * 2 * kHalf;
#pragma unroll
            for (int i = 0; i < kTurns; ++i) {
                const int r = kChunks <= 32 ? i * (32 / kChunks) + lane / kChunks : i / (kChunks / 32);
                const int c = kChunks <= 32 ? lane % kChunks : (i % (kChunks / 32)) * 32 + lane;
                const int from = __shfl_sync(0xffffffffu, row, r);
                const bool ok = from >= 0 && c < cpr;
                const int64_t byte = ok ? (int64_t)from * (a.cache.D * (int)sizeof(C)) + c * 16 : 0;
                const uint32_t at = to + r * kPitch + ((c ^ (r & 7)) << 4);
                copy16(at, static_cast<const char *>(a.cache.k) + byte, ok);
                copy16(at + kHalf, static_cast<const char *>(a.cache.v) + byte, ok);
            }
            if constexpr (kScaled) {
                uint8_t *x = scales + slot * 2 * KEYS;
                if (lane < KEYS) {
                    x[lane] = (uint8_t)sk;
                    x[KEYS + lane] = (uint8_t)sv;
                }
            }
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
        resolve(s + 1);
        look(s + 2);
    }
    // The oldest slot on its way is complete and seen by the warp.
    __device__ __forceinline__ void ready() {
        copies_wait<STAGES - 2>();
        __syncwarp();
    }
};

}  // namespace attn
}  // namespace kda
