// Attention over a paged cache (kda_attention.h), what its kernels share: how the work is cut, how keys and values
// stream in, and how the pieces of one result are joined.
//
// An item is one (sequence, block of query rows, key head); its keys are cut into units of 8, 16 or 32 (by the kernel).
// All items' units, one after another, are dealt out in equal shares to the workers of the grid: warps, each with its own
// ring of shared memory and no barrier with the others, or, where there are many query rows, teams of warps that
// share a ring and take some of the rows each. A worker has at most one item that began in the share before and one that
// goes on in the next; such pieces leave (m, l, O) in scratch: the reference m of their exponentials 2^(s - m), the
// sum l of those, and O = sum 2^(s - m) v. A second kernel joins them in the order of the workers. Which items are cut follows
// from the lengths and sizes alone, so results repeat bit for bit.
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
// What an item costs beside its units, in units, when the work is dealt out: its queries in, its result out and the waits in
// between. (16 sequences of up to 8192 tokens, among them one of 4 and one at rest, four new tokens each: 51 us without it, the
// short ones' items one after another in two shares, and 44 with it; 256 sequences of up to 900 tokens 56 and 50.)
constexpr uint32_t kItemCost = 2;
constexpr int kThreads = 32 * kWarps;

struct Args {
    const void *q;
    void *o;
    float *lse;
    int64_t q_stride;
    int B, T, Hq, group;
    uint32_t group_magic;  // ceil(2^32 / group): row / group is the upper half of row * group_magic while row * group < 2^32
    int rows;              // query rows of an item (at most)
    int row_blocks, per_seq;  // items of a sequence: blocks of query rows * key heads
    int unit_shift;        // keys of a unit, as a power of two
    int workers;
    float scale_log2;      // scale * log2 e
    Cache cache;
    float *pieces;         // [2 workers][rows * (D + 2)]: O [rows][D], then (m, l) [rows]
    int2 *ends;            // of each item (in the order of the deal): the workers that have its first and its last piece
};

__device__ __forceinline__ int token_of(const Args &a, int row) {
    return a.group == 1 ? row : (int)__umulhi((uint32_t)row, a.group_magic);
}
__device__ __forceinline__ uint32_t units_of(const Args &a, int len) {
    const uint32_t n = ((uint32_t)len + (1u << a.unit_shift) - 1) >> a.unit_shift;
    return n == 0 ? 1 : n;
}

// The units and costs of an item.
__device__ __forceinline__ uint32_t weight_of(const Args &a, int len) { return units_of(a, len) + kItemCost; }

// The weights of all items (below 2^32, checked on the host for the longest sequences) dealt out: how many workers have a
// share (each then has some), and where share w begins.
struct Deal {
    uint32_t n, base, more;  // the first `more` shares have base + 1 units
    __device__ __forceinline__ Deal(const Args &a, uint32_t total) {
        n = total < (uint32_t)a.workers ? total : (uint32_t)a.workers;
        base = total / n;
        more = total - base * n;
    }
    __device__ __forceinline__ uint32_t start(uint32_t w) const { return w * base + (w < more ? w : more); }
};

// A scan over the sequences by the threads of a block: thread i adds up the sequences i * each .. i * each + each - 1.
struct Scan {
    int each, first;
    uint32_t sum, before, total;  // weights of the thread's sequences, of those before, of all
};
// `mem`: an int for each warp.
__device__ __forceinline__ Scan scan_sequences(const Args &a, uint32_t *mem) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, threads = blockDim.x;
    Scan s;
    s.each = (a.B + threads - 1) / threads;
    s.first = threadIdx.x * s.each;
    s.sum = 0;
#pragma unroll 1
    for (int b = s.first; b < s.first + s.each && b < a.B; ++b) s.sum += weight_of(a, cache_len(a.cache, b));
    s.sum *= a.per_seq;
    uint32_t scan = s.sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += x;
    }
    if (lane == 31) mem[warp] = scan;
    __syncthreads();
    s.before = scan - s.sum;
    s.total = 0;
#pragma unroll 1
    for (int v = 0; v < threads / 32; ++v) {
        if (v < warp) s.before += mem[v];
        s.total += mem[v];
    }
    return s;
}

// One piece of work: units u0 .. u1 - 1 of an item's `units` (none where the share's border falls into the item's cost, which
// stands before its units), and what they weigh.
struct Piece {
    int b, len, head, row0, rows;  // first query row of the item and how many it has
    uint32_t u0, u1, units, weight;
    __device__ __forceinline__ bool none() const { return u0 == u1; }
    int last;  // keys that the last of its rows sees: no key at or after this one counts
    __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == units; }
    // The piece for `most` of its rows from row `from` on (none: `last` 0).
    __device__ __forceinline__ void mine(const Args &a, int from, int most);
};
__device__ __forceinline__ int seen(const Args &a, int len, int row) {
    const int n = len - a.T + token_of(a, row) + 1;
    return n < 0 ? 0 : n;
}

__device__ __forceinline__ void Piece::mine(const Args &a, int from, int most) {
    row0 += from;
    rows = rows - from < most ? rows - from : most;
    last = rows > 0 ? seen(a, len, row0 + rows - 1) : 0;
}

// A worker's way through its share, piece by piece: items in the order (sequence, block of rows, key head).
struct Walk {
    int b, len, rb, head;
    uint32_t w0, left;  // weight of the item that is done, and of the share that is left
    int next_len;  // of sequence b + 1, read ahead
    __device__ __forceinline__ void read_ahead(const Args &a) { next_len = b + 1 < a.B ? cache_len(a.cache, b + 1) : 0; }
    __device__ __forceinline__ Piece piece(const Args &a) const {
        Piece p;
        p.b = b;
        p.len = len;
        p.units = units_of(a, len);
        p.weight = p.units + kItemCost - w0;
        p.weight = left < p.weight ? left : p.weight;
        const uint32_t w1 = w0 + p.weight;
        p.u0 = w0 < kItemCost ? 0 : w0 - kItemCost;
        p.u1 = w1 < kItemCost ? 0 : w1 - kItemCost;
        p.head = head;
        p.row0 = rb * a.rows;
        const int all = a.T * a.group;
        p.rows = all - p.row0 < a.rows ? all - p.row0 : a.rows;
        p.last = seen(a, len, p.row0 + p.rows - 1);
        return p;
    }
    // On past a piece.
    __device__ __forceinline__ void step(const Args &a, uint32_t weight) {
        left -= weight;
        w0 = 0;
        if (++head < a.cache.heads) return;
        head = 0;
        if (++rb < a.row_blocks) return;
        rb = 0;
        ++b;
        len = next_len;
        read_ahead(a);
    }
};
// The start of the share of every warp's worker (of TEAM warps); `mem`: 3 kWarps ints. Ends with a barrier; `left` 0: no share.
template <int TEAM>
__device__ __forceinline__ Walk find_walk(const Args &a, uint32_t *mem) {
    const Scan sc = scan_sequences(a, mem);
    const Deal deal(a, sc.total);
    const uint32_t w0 = blockIdx.x * (kWarps / TEAM);
    uint32_t *found = mem + kWarps, *rest = found + kWarps;
#pragma unroll 1
    for (uint32_t v = 0; v < kWarps / TEAM && w0 + v < deal.n; ++v) {
        const uint32_t at = deal.start(w0 + v);
        if (at - sc.before < sc.sum) {  // one thread's
            int b = sc.first;
            uint32_t before = sc.before;
#pragma unroll 1
            for (;;) {
                const uint32_t x = weight_of(a, cache_len(a.cache, b)) * a.per_seq;
                if (at - before < x) break;
                before += x;
                ++b;
            }
            found[v] = b;
            rest[v] = at - before;
        }
    }
    __syncthreads();
    const uint32_t v = (threadIdx.x >> 5) / TEAM;
    Walk k;
    k.left = 0;
    k.b = k.len = k.rb = k.head = k.w0 = k.next_len = 0;
    if (w0 + v < deal.n) {
        k.left = deal.start(w0 + v + 1) - deal.start(w0 + v);
        k.b = (int)found[v];
        k.len = cache_len(a.cache, k.b);
        const uint32_t weight = weight_of(a, k.len), item = rest[v] / weight;
        k.rb = (int)(item / a.cache.heads);
        k.head = (int)item - k.rb * a.cache.heads;
        k.w0 = rest[v] - item * weight;
        k.read_ahead(a);
    }
    return k;
}
constexpr int kPlanBytes = 4 * kWarps * 4;

// Offsets (elements) of a query row in q, and of its row in o and lse.
__device__ __forceinline__ int64_t q_at(const Args &a, const Piece &p, int r) {
    const int row = p.row0 + r, t = token_of(a, row);
    return ((int64_t)p.b * a.T + t) * a.q_stride + (int64_t)(p.head * a.group + row - t * a.group) * a.cache.D;
}
__device__ __forceinline__ int64_t out_row(const Args &a, const Piece &p, int r) {
    const int row = p.row0 + r, t = token_of(a, row);
    return ((int64_t)p.b * a.T + t) * a.Hq + p.head * a.group + row - t * a.group;
}
// A worker's scratch for a piece: the first when the item began before, the second when it goes on (or both).
__device__ __forceinline__ float *piece_mem(const Args &a, int worker, bool begins) {
    return a.pieces + (int64_t)(2 * worker + (begins ? 1 : 0)) * a.rows * (a.cache.D + 2);
}

// The workers of the item's ends, one thread's to say.
__device__ __forceinline__ void tell_ends(const Args &a, const Piece &p, int worker) {
    int2 *at = a.ends + (int64_t)p.b * a.per_seq + p.row0 / a.rows * a.cache.heads + p.head;
    if (p.u0 == 0) at->x = worker;
    if (p.u1 == p.units) at->y = worker;
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

// The stream of a worker's keys and values, through a ring of SLOTS slots of shared memory: K of a unit, V of it, K of the
// next one, and so on, so that half a unit is enough to keep and the rest of the ring is on its way. A slot holds KEYS
// rows of kPitch bytes, 16-byte chunk c of row r at chunk c ^ (r & 7): 8 rows at one chunk lie in different banks.
// Rows that no query of the piece sees, or without a page, are zeros. The stream runs ahead of the computation over the
// borders of pieces. The page of a row is read from the table two units before its copies are issued, and the rows'
// exponent bytes one unit before, so that neither is waited for.
// Of a team, each warp copies its part of every unit's rows, and a barrier of the team in front of each slot both shows its
// rows to all and says that the slot before is free.
template <typename C, int DP, int KEYS, int SLOTS, int TEAM = 1>
struct Stream {
    static constexpr int kPitch = DP * (int)sizeof(C) < 128 ? 128 : DP * (int)sizeof(C);
    static constexpr int kSlot = KEYS * kPitch;
    static constexpr int kBytes = SLOTS * kSlot;
    static constexpr int kUnits = SLOTS / 2 + 2;  // whose exponent bytes may be held at a time
    static constexpr int kScaleBytes = sizeof(C) == 1 ? kUnits * 2 * KEYS : 0;
    static constexpr int kChunks = kPitch / 16;         // of a row
    static constexpr int kMine = KEYS / TEAM;           // rows that a warp copies
    static constexpr int kTurns = kMine * kChunks / 32;
    static_assert(kTurns >= 1 && (TEAM == 1 || kMine % 4 == 0), "whole turns");
    static constexpr bool kScaled = sizeof(C) == 1;

    const Args &a;
    uint32_t ring;           // shared address
    uint8_t *scales;         // [kUnits][2][KEYS] exponent bytes
    int lane;
    Walk walk;               // of the unit that is looked up next
    uint32_t u, u1, weight;  // that unit, where its piece ends, what the piece weighs
    int last;                // keys of its piece that count
    int entry, place;        // of this lane's row (first + lane % kMine), looked up: the table's entry, the row within the page and head (-1: none)
    int row;                 // and of the unit that is copied next: the row of the cache (-1: zeros)
    uint32_t sk, sv;         // its exponent bytes
    int slot, unit_in, unit_out;  // the oldest slot, and where exponent bytes are written and read
    int first, barrier;           // team: the first row that this warp copies, the team's barrier
    bool begun;

    __device__ __forceinline__ Stream(const Args &a_, unsigned char *mem, uint8_t *sc, int lane_, int warp, const Walk &w)
        : a(a_), ring(smem_u32(mem)), scales(sc), lane(lane_), walk(w), sk(0), sv(0), slot(0), unit_in(0), unit_out(0),
          first(warp % TEAM * kMine), barrier(1 + warp / TEAM), begun(false) {
        enter();
        place = -1;
        // one unit looked up, then one resolved and the next looked up; then the slots in order
#pragma unroll 1
        for (int i = -2; i < SLOTS; ++i) {
            if (i < 0 || (i & 1)) {
                if (i > 0) copy_rows(a.cache.v, i);
                resolve();
                look();
            } else {
                fetch_k(i);
            }
        }
    }
    __device__ __forceinline__ void enter() {
        while (walk.left != 0) {
            const Piece p = walk.piece(a);
            u = p.u0;
            u1 = p.u1;
            last = p.last;
            weight = p.weight;
            if (!p.none()) break;
            walk.step(a, weight);
        }
    }
    __device__ __forceinline__ void look() {
        place = -1;
        if (walk.left == 0) return;
        const int pos = (int)u * KEYS + first + (lane & (kMine - 1));
        if (pos < last) {
            int at, s;
            cache_split(a.cache, pos, at, s);
            entry = a.cache.table[(int64_t)walk.b * a.cache.table_stride + at];
            place = walk.head * a.cache.page + s;
        }
        if (++u == u1) {
            walk.step(a, weight);
            enter();
        }
    }
    __device__ __forceinline__ void resolve() {
        row = -1;
        sk = sv = 0;  // not those of another sequence's row, which may be no number
        if (place < 0) return;
        if ((unsigned)entry < (unsigned)a.cache.pages) {
            row = entry * (int)a.cache.page_rows + place;
            if constexpr (kScaled) {
                const int64_t x = (int64_t)entry * a.cache.scale_stride + place;
                sk = a.cache.ks[x];
                sv = a.cache.vs[x];
            }
        } else {
            atomicOr(a.cache.err, kDeviceErrCache);
        }
    }
    __device__ __forceinline__ void copy_rows(const void *base, int to_slot) {
        const uint32_t to = ring + to_slot * kSlot + first * kPitch;
        const uint32_t width = a.cache.D * (uint32_t)sizeof(C);
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int r = kChunks <= 32 ? i * (32 / kChunks) + lane / kChunks : i / (kChunks / 32);
            const int c = kChunks <= 32 ? lane % kChunks : (i % (kChunks / 32)) * 32 + lane;
            const int from = __shfl_sync(0xffffffffu, row, r);
            const bool ok = from >= 0 && c * 16u < width;
            copy16(to + r * kPitch + ((c ^ ((first + r) & 7)) << 4), static_cast<const char *>(base) + (uint64_t)(uint32_t)(ok ? from : 0) * width + (ok ? c * 16u : 0u), ok);
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    }
    __device__ __forceinline__ void fetch_k(int to_slot) {
        copy_rows(a.cache.k, to_slot);
        if constexpr (kScaled) {
            uint8_t *x = scales + unit_in * 2 * KEYS;
            if (lane < kMine) {
                x[first + lane] = (uint8_t)sk;
                x[KEYS + first + lane] = (uint8_t)sv;
            }
            unit_in = unit_in == kUnits - 1 ? 0 : unit_in + 1;
        }
    }
    __device__ __forceinline__ void fetch_v(int to_slot) {
        copy_rows(a.cache.v, to_slot);
        resolve();
        look();
    }
    // What comes SLOTS slots after slot `at`, which held K or V (`V`), goes into it.
    template <bool V>
    __device__ __forceinline__ void refill(int at) {
        if constexpr (V == (SLOTS % 2 == 0))
            fetch_v(at);
        else
            fetch_k(at);
    }
    // The oldest slot, K or V, is complete and seen by the worker. A team is then done with the slot before.
    template <bool V>
    __device__ __forceinline__ void ready() {
        if constexpr (TEAM == 1) {
            copies_wait<SLOTS - 1>();
            __syncwarp();
        } else {
            copies_wait<SLOTS - 2>();
            tcu::bar_named(barrier, 32 * TEAM);
            if (begun) refill<!V>(slot == 0 ? SLOTS - 1 : slot - 1);
            begun = true;
        }
    }
    // Shared address of the oldest slot; the exponent bytes of the oldest unit.
    __device__ __forceinline__ uint32_t oldest() const { return ring + slot * kSlot; }
    __device__ __forceinline__ const uint8_t *bytes() const { return scales + unit_out * 2 * KEYS; }
    // The warp is done with the oldest slot, K or V.
    template <bool V>
    __device__ __forceinline__ void release() {
        if constexpr (TEAM == 1) {
            __syncwarp();
            refill<V>(slot);
        }
        slot = slot == SLOTS - 1 ? 0 : slot + 1;
        if constexpr (V) unit_out = unit_out == kUnits - 1 ? 0 : unit_out + 1;
    }
};

}  // namespace attn
}  // namespace kda
