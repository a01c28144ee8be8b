// Attention over a paged cache (kda_attention.h), what its kernels share: how the work is cut, how keys and values
// stream in, and how the pieces of one result are joined.
//
// An item is one (sequence, block of query rows, key head); its keys are cut into units of UNIT (16 or 32, by the kernel).
// All items' units, one after another, are dealt out in equal shares to the warps of the grid: a warp is a worker of its
// own, with its own ring of shared memory and no barrier with the others. It has at most one item that began in the
// share before and one that goes on in the next; such pieces leave (m, l, O) in scratch: the reference m of their
// exponentials 2^(s - m), the sum l of those, and O = sum 2^(s - m) v. A second kernel joins them in the order of
// the workers. Which items are cut follows from the lengths and sizes alone, so results repeat bit for bit.
// (Blocks of four warps that shared each item's keys and joined them in shared memory: 4 to 7 us for every piece
// of an item, most of it waiting; 2048 items of 450 keys took 74 us.)
//
// Query rows of an item are the (token, head of the group) pairs t * group + g of one key head, in blocks of
// `rows`; the keys that a row sees are those at positions below len - T + t + 1.
#pragma once

#include "cache_common.cuh"

namespace kda {
namespace attn {

using namespace mix;

constexpr int kWarps = 4;  // of a block
constexpr int kThreads = 32 * kWarps;

struct Args {
    const void *q;
    void *o;
    float *lse;
    int64_t q_stride;
    int B, T, Hq, group;
    int rows;          // query rows of an item (at most)
    int per_seq;       // items of a sequence: blocks of query rows * key heads
    int unit;          // keys of a unit
    int workers;
    float scale_log2;  // scale * log2 e
    Cache cache;
    float *pieces;     // [2 workers][rows * (D + 2)]: O [rows][D], then (m, l) [rows]
};

__device__ __forceinline__ int units_of(int len, int unit) { return len <= unit ? 1 : (len + unit - 1) / unit; }

// How many workers have a share (each then has a unit at least), the first unit of share w, and whose share unit x is in.
__device__ __forceinline__ int sharers(const Args &a, int64_t total) { return total < a.workers ? (int)total : a.workers; }
__device__ __forceinline__ int64_t share(int64_t total, int w, int n) { return total * w / n; }
__device__ __forceinline__ int owner(int64_t total, int64_t x, int n) { return (int)(((x + 1) * n - 1) / total); }

// A scan over the sequences by the NT threads of a block: thread i adds up the sequences i * each .. i * each + each - 1.
template <int NT>
struct Scan {
    int each, first;
    int64_t sum, before, total;  // units of the thread's sequences, of those before, of all
    // `mem`: NT / 32 int64
    __device__ __forceinline__ void run(const Args &a, int64_t *mem) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        each = (a.B + NT - 1) / NT;
        first = threadIdx.x * each;
        sum = 0;
        for (int b = first; b < first + each && b < a.B; ++b) sum += units_of(cache_len(a.cache, b), a.unit);
        sum *= a.per_seq;
        int64_t scan = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += x;
        }
        if (lane == 31) mem[warp] = scan;
        __syncthreads();
        before = scan - sum;
        total = 0;
#pragma unroll
        for (int v = 0; v < NT / 32; ++v) {
            if (v < warp) before += mem[v];
            total += mem[v];
        }
    }
};

// One piece of work: units u0 .. u1 - 1 of an item's `units`.
struct Piece {
    int b, len, head, row0, rows;  // first query row of the item and how many it has
    int u0, u1, units;
    int last;  // keys that the last of its rows sees: no key at or after this one counts
    __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == units; }
};
__device__ __forceinline__ int seen(const Args &a, int len, int row) {
    const int n = len - a.T + row / a.group + 1;
    return n < 0 ? 0 : n;
}
__device__ __forceinline__ Piece piece_of(const Args &a, int b, int len, int item, int u0, int64_t left) {
    Piece p;
    p.b = b;
    p.len = len;
    p.units = units_of(len, a.unit);
    p.u0 = u0;
    p.u1 = left < p.units - u0 ? u0 + (int)left : p.units;
    const int rb = item / a.cache.heads;
    p.head = item - rb * a.cache.heads;
    p.row0 = rb * a.rows;
    const int all = a.T * a.group;
    p.rows = all - p.row0 < a.rows ? all - p.row0 : a.rows;
    p.last = seen(a, len, p.row0 + p.rows - 1);
    return p;
}

// A worker's way through its share, piece by piece.
struct Walk {
    int b, len, item, u0, next_len;  // next_len: of sequence b + 1, read ahead
    int64_t left;
    __device__ __forceinline__ void read_ahead(const Args &a) { next_len = b + 1 < a.B ? cache_len(a.cache, b + 1) : 0; }
    __device__ __forceinline__ Piece piece(const Args &a) const { return piece_of(a, b, len, item, u0, left); }
    __device__ __forceinline__ void step(const Args &a, const Piece &p) {
        left -= p.u1 - p.u0;
        u0 = 0;
        if (++item == a.per_seq) {
            item = 0;
            ++b;
            len = next_len;
            read_ahead(a);
        }
    }
};
// The start of every warp's share; `mem`: 2 kWarps int64 each. Ends with a barrier; `left` 0: no share.
__device__ __forceinline__ Walk find_walk(const Args &a, int64_t *mem) {
    Scan<kThreads> sc;
    sc.run(a, mem);
    const int n = sharers(a, sc.total), w0 = blockIdx.x * kWarps;
    int64_t *found = mem + kWarps;  // [kWarps]: sequence in the upper half, and (u0 + units * item) fits the lower
    int64_t *rest = found + kWarps;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) {
        if (w0 + v >= n) break;
        const int64_t at = share(sc.total, w0 + v, n);
        if (at >= sc.before && at < sc.before + sc.sum) {  // one thread's
            int b = sc.first;
            int64_t before = sc.before;
            for (;;) {
                const int64_t x = (int64_t)units_of(cache_len(a.cache, b), a.unit) * a.per_seq;
                if (at < before + x) break;
                before += x;
                ++b;
            }
            found[v] = b;
            rest[v] = at - before;
        }
    }
    __syncthreads();
    const int v = threadIdx.x >> 5;
    Walk k;
    k.left = 0;
    k.b = k.len = k.item = k.u0 = k.next_len = 0;
    if (w0 + v < n) {
        k.left = share(sc.total, w0 + v + 1, n) - share(sc.total, w0 + v, n);
        k.b = (int)found[v];
        k.len = cache_len(a.cache, k.b);
        const int units = units_of(k.len, a.unit);
        k.item = (int)(rest[v] / units);
        k.u0 = (int)(rest[v] - (int64_t)k.item * units);
        k.read_ahead(a);
    }
    return k;
}
constexpr int kPlanBytes = 3 * kWarps * 8;

// Offsets (elements) of a query row in q, and of its row in o and lse.
__device__ __forceinline__ int64_t q_at(const Args &a, const Piece &p, int r) {
    const int row = p.row0 + r, t = row / a.group;
    return ((int64_t)p.b * a.T + t) * a.q_stride + (int64_t)(p.head * a.group + row - t * a.group) * a.cache.D;
}
__device__ __forceinline__ int64_t out_row(const Args &a, const Piece &p, int r) {
    const int row = p.row0 + r, t = row / a.group;
    return ((int64_t)p.b * a.T + t) * a.Hq + p.head * a.group + row - t * a.group;
}
// A worker's scratch for a piece: the first when the item began before, the second when it goes on (or both).
__device__ __forceinline__ float *piece_mem(const Args &a, int worker, bool begins) {
    return a.pieces + (int64_t)(2 * worker + (begins ? 1 : 0)) * a.rows * (a.cache.D + 2);
}

constexpr float kLn2 = 0.6931471805599453f;
// log of a row's sum of e^score from the reference m (base 2) and the sum l
__device__ __forceinline__ float lse_of(float m, float l) { return l > 0.f ? (m + log2f(l)) * kLn2 : (l == 0.f ? -INFINITY : l); }

// The next kernel of the stream may be set up while this one runs, and there it waits for this one's results.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// 16 bytes of a row of the cache into shared memory, zeros where `ok` is false.
__device__ __forceinline__ void copy16(uint32_t to, const void *from, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(to), "l"(from), "r"(ok ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// The stream of a worker's keys and values, through a ring of STAGES slots of shared memory. A slot holds a unit: KEYS rows of K
// and of V, kPitch bytes each, 16-byte chunk c of row r at chunk c ^ (r & 7): 8 rows at one chunk lie in
// different banks. Rows that no query of the piece sees, or without a page, are zeros. It runs ahead of the
// computation over the borders of pieces. The page of a row is read from the table two units before its copies are
// issued, and the rows' exponent bytes one unit before, so that neither is waited for.
template <typename C, int DP, int KEYS, int STAGES>
struct Stream {
    static constexpr int kPitch = DP * (int)sizeof(C) < 128 ? 128 : DP * (int)sizeof(C);
    static constexpr int kHalf = KEYS * kPitch;  // K or V of a slot
    static constexpr int kBytes = STAGES * 2 * kHalf;
    static constexpr int kScaleBytes = STAGES * 2 * KEYS;
    static constexpr int kChunks = kPitch / 16;            // of a row
    static constexpr int kTurns = KEYS * kChunks / 32;     // copies of a lane for KEYS rows
    static constexpr bool kScaled = sizeof(C) == 1;

    const Args &a;
    uint32_t ring;         // shared address
    uint8_t *scales;       // [STAGES][2][KEYS] exponent bytes
    int lane;
    Walk walk;             // of the unit that is looked up next
    Piece p;
    int u;
    int entry, place;      // of this lane's row (lane % KEYS), looked up: the table's entry, the row within the page and head (-1: none)
    int row;               // and of the unit before that: the row of the cache (-1: zeros)
    uint32_t sk, sv;       // its exponent bytes

    __device__ __forceinline__ Stream(const Args &a_, unsigned char *mem, uint8_t *sc, int lane_, const Walk &w)
        : a(a_), ring(smem_u32(mem)), scales(sc), lane(lane_), walk(w), sk(0), sv(0) {
        if (walk.left > 0) {
            p = walk.piece(a);
            u = p.u0;
        }
        look();
        resolve();
        look();
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) fetch(i);
    }
    __device__ __forceinline__ void look() {
        place = -1;
        if (walk.left <= 0) return;
        const int pos = u * KEYS + (lane & (KEYS - 1));
        if (pos < p.last) {
            int at, slot;
            cache_split(a.cache, pos, at, slot);
            entry = a.cache.table[(int64_t)p.b * a.cache.table_stride + at];
            place = p.head * a.cache.page + slot;
        }
        if (++u == p.u1) {
            walk.step(a, p);
            if (walk.left > 0) {
                p = walk.piece(a);
                u = p.u0;
            }
        }
    }
    __device__ __forceinline__ void resolve() {
        row = -1;
        if (place < 0) return;
        if ((unsigned)entry < (unsigned)a.cache.pages) {
            row = (int)((int64_t)entry * a.cache.page_rows) + place;
            if constexpr (kScaled) {
                const int64_t x = (int64_t)entry * a.cache.scale_stride + place;
                sk = a.cache.ks[x];
                sv = a.cache.vs[x];
            }
        } else {
            atomicOr(a.cache.err, kDeviceErrCache);
        }
    }
    __device__ __forceinline__ void fetch(int slot) {
        const int width = a.cache.D * (int)sizeof(C);
        const uint32_t to = ring + slot * 2 * kHalf;
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int r = kChunks <= 32 ? i * (32 / kChunks) + lane / kChunks : i / (kChunks / 32);
            const int c = kChunks <= 32 ? lane % kChunks : (i % (kChunks / 32)) * 32 + lane;
            const int from = __shfl_sync(0xffffffffu, row, r);
            const bool ok = from >= 0 && c * 16 < width;
            const int64_t byte = ok ? (int64_t)from * width + c * 16 : 0;
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
        asm volatile("cp.async.commit_group;\n" ::: "memory");
        resolve();
        look();
    }
    // The oldest slot on its way is complete and seen by the warp.
    __device__ __forceinline__ void ready() {
        copies_wait<STAGES - 2>();
        __syncwarp();
    }
    // The warp is done with slot `slot`, the oldest: the next unit goes into the one before it. Returns the new oldest.
    __device__ __forceinline__ int next(int slot) {
        __syncwarp();
        fetch(slot == 0 ? STAGES - 1 : slot - 1);
        return slot == STAGES - 1 ? 0 : slot + 1;
    }
};

}  // namespace attn
}  // namespace kda
