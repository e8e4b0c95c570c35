// What the operators on the paged key/value cache share: the step's sequences
// as the device sees them, with every index from device memory checked before
// it is used, and the division of the attention's work between workers.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace bitlinear {

// Beside FaultCode's bits of the fault word: a sequence, length or page index in
// device memory out of range.
constexpr unsigned int FAULT_BAD_INDEX = 2;

namespace paged {

// The step's sequences (see bitlinear_seqs). tokens is the number of query
// rows that exist; the arrays live in device memory, so their values are only
// known there.
struct Seqs {
    const int *q_start;    // [seqs + 1]
    const int *kv_len;     // [seqs]
    const int *table;      // [seqs][table_cols]
    int seqs;
    int table_cols;
    int tokens;
    int page_shift;        // log2 of the page size
    int pages;             // pages of the cache
};

__device__ __forceinline__ void fault_index() { atomicOr(&g_fault_word, FAULT_BAD_INDEX); }

// One sequence: rows q0 .. q0 + qlen, the last of them at position kv - 1.
struct View {
    int q0, qlen, kv;
};

// Sequence s, cut to the rows and the page slots that exist. False when a value
// lay outside them.
__device__ __forceinline__ bool read_view(const Seqs &q, int s, View &v)
{
    const int b = __ldg(q.q_start + s), e = __ldg(q.q_start + s + 1), n = __ldg(q.kv_len + s);
    v.q0 = min(max(b, 0), q.tokens);
    v.qlen = min(max(e, v.q0), q.tokens) - v.q0;
    v.kv = min(max(n, 0), q.table_cols << q.page_shift);
    return v.q0 == b && v.q0 + v.qlen == e && v.kv == n;
}

// The same for reading, where the cut sequence will do; a value outside is recorded
// as a fault.
__device__ __forceinline__ View view(const Seqs &q, int s)
{
    View v;
    if (!read_view(q, s, v))
        fault_index();
    return v;
}

// Page of table column c of sequence s, or -1 (recorded as a fault) when the
// table holds no page of the cache there.
__device__ __forceinline__ int page_of(const Seqs &q, int s, int c)
{
    const int id = __ldg(q.table + static_cast<int64_t>(s) * q.table_cols + c);
    if (id >= 0 && id < q.pages)
        return id;
    fault_index();
    return -1;
}

// ---------------------------------------------------------------- schedule
//
// The attention's work is cut into items: item_rows consecutive rows of one
// sequence and key head, where row r is query head r % group of token r / group, so the
// query heads that share a key head share its tiles. An item takes `full` units
// per tile of BN keys that any of its rows sees, or `half` when it has no more
// than half its rows, and `start` units ahead of its first tile's. All units of a
// launch, items in order and key heads outermost, are dealt to the workers in equal
// contiguous runs; a tile belongs to the run that it begins in: a long sequence is
// split wherever a run ends, and a batch of ragged ones stays balanced without the
// host knowing a length. A worker that gets a whole item writes its output;
// otherwise it leaves a partial sum that is joined in the order of the keys.

// Division of row numbers by a launch constant: n / d for 0 <= n < 2^31 is the
// high word of n * mul shifted (mul = ceil(2^(31 + s) / d), s = ceil(log2 d):
// the excess of mul d over 2^(31 + s) is below 2^s, so the quotient is exact).
struct Divide {
    uint32_t mul;
    int shift;             // -1: d is 1

    __device__ __forceinline__ int operator()(int n) const
    {
        return shift < 0 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), mul) >> shift);
    }
};

struct Work {
    Seqs seqs;
    Divide by_group;
    int group;             // query heads per key head
    int kv_heads;
    int item_rows;         // rows of an item
    int full, half;        // units of a tile
    int start;             // and of an item besides those of its tiles
    int window;            // 0: none
    int min_rows, max_rows;  // sequences of this launch: min_rows <= qlen * group <= max_rows
};

constexpr int MAX_GROUPS = 512;          // of 32 sequences: at most 16384 sequences

struct Tiles {
    int begin, end;        // key tiles
    int klo, khi;          // keys that any row of the item sees
};

// The k-th item of a sequence of n: the rows nearest its end, which see the most
// keys, take turns with those nearest its beginning, so that a run of units
// never holds many short items.
__device__ __forceinline__ int item_at(int k, int n) { return (k & 1) ? k >> 1 : n - 1 - (k >> 1); }

__device__ __forceinline__ int items_of(const Work &w, const View &v)
{
    return static_cast<int>(static_cast<unsigned>(v.qlen * w.group + w.item_rows - 1) /
                            static_cast<unsigned>(w.item_rows));
}

// Key tiles of rows m * item_rows .. of a sequence.
template <int BN>
__device__ __forceinline__ Tiles item_tiles(const Work &w, const View &v, int m)
{
    const int r1 = min((m + 1) * w.item_rows, v.qlen * w.group) - 1;
    const int first = v.kv - v.qlen + w.by_group(m * w.item_rows);   // position of the first row
    const int last = v.kv - v.qlen + w.by_group(r1);
    Tiles t;
    t.khi = max(last + 1, 0);
    t.klo = w.window > 0 ? max(first - w.window + 1, 0) : 0;
    t.begin = t.klo / BN;
    // rows before position 0 see nothing; they still take one unit, which
    // writes their zeros
    t.end = max((t.khi + BN - 1) / BN, t.begin + 1);
    return t;
}

__device__ __forceinline__ bool in_launch(const Work &w, const View &v)
{
    const int rows = v.qlen * w.group;
    return rows >= w.min_rows && rows <= w.max_rows;
}

__device__ __forceinline__ int64_t warp_sum(int64_t n)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        n += __shfl_xor_sync(0xffffffffu, n, o);
    return n;
}

// sum of the lanes up to this one
__device__ __forceinline__ int64_t warp_scan(int64_t n)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, n, o);
        if (lane >= o)
            n += x;
    }
    return n;
}

__device__ __forceinline__ int tile_units(const Work &w, const View &v, int m)
{
    return v.qlen * w.group - m * w.item_rows > w.item_rows / 2 ? w.full : w.half;
}

// Units of the 32 sequences of group g, one per lane (the whole warp). A
// sequence of several items has them counted by all lanes.
template <int BN>
__device__ __forceinline__ int64_t seq_units(const Work &w, int g)
{
    const int lane = threadIdx.x & 31;
    const int s = g * 32 + lane;
    View v{};
    if (s < w.seqs.seqs) {
        v = view(w.seqs, s);
        if (!in_launch(w, v))
            v.qlen = 0;
    }
    const bool many = v.qlen * w.group > w.item_rows;
    int64_t n = 0;
    if (v.qlen > 0 && !many) {
        const Tiles t = item_tiles<BN>(w, v, 0);
        n = (t.end - t.begin) * tile_units(w, v, 0) + w.start;
    }
    for (unsigned left = __ballot_sync(0xffffffffu, many); left != 0; left &= left - 1) {
        const int at = __ffs(left) - 1;
        View x;
        x.q0 = 0;
        x.qlen = __shfl_sync(0xffffffffu, v.qlen, at);
        x.kv = __shfl_sync(0xffffffffu, v.kv, at);
        int64_t sum = 0;
        for (int m = lane; m * w.item_rows < x.qlen * w.group; m += 32) {
            const Tiles t = item_tiles<BN>(w, x, m);
            sum += (t.end - t.begin) * tile_units(w, x, m) + w.start;
        }
        sum = warp_sum(sum);
        if (lane == at)
            n = sum;
    }
    return n;
}

// A tile of the launch: the item and the tile inside it.
template <int BN>
struct Cursor {
    int h, s, k, m, tile;  // k-th item of the sequence: rows m * w.item_rows ..
    int units;             // of each of its tiles
    View v;
    Tiles t;

    __device__ __forceinline__ void open(const Work &w)
    {
        m = item_at(k, items_of(w, v));
        t = item_tiles<BN>(w, v, m);
        units = tile_units(w, v, m);
        tile = t.begin;
    }

    // The first tile of the next item. Only called while units are left, so a
    // sequence of this launch is always found.
    __device__ __forceinline__ void next_item(const Work &w)
    {
        if (++k * w.item_rows >= v.qlen * w.group) {
            k = 0;
            do {
                if (++s == w.seqs.seqs) {
                    s = 0;
                    ++h;
                }
                v = view(w.seqs, s);
            } while (!in_launch(w, v));
        }
        open(w);
    }

    // Moves to the item that holds unit `off` of the 32 sequences of group g,
    // whose units n the lanes hold (the whole warp), and to its first tile that
    // begins there or behind. Returns how far behind; the tile may be the one
    // after the item's last.
    __device__ __forceinline__ int seek(const Work &w, int g, int64_t n, int64_t off)
    {
        const int lane = threadIdx.x & 31;
        const int64_t upto = warp_scan(n);
        const int at = __ffs(__ballot_sync(0xffffffffu, off < upto)) - 1;
        off -= __shfl_sync(0xffffffffu, upto - n, at);
        s = g * 32 + at;
        v = view(w.seqs, s);
        k = 0;
        // the item, 32 of the sequence's at a time
        const int items = items_of(w, v);
        for (int k0 = 0; items > 1; k0 += 32) {
            int64_t c = 0;
            if (k0 + lane < items) {
                const Tiles x = item_tiles<BN>(w, v, item_at(k0 + lane, items));
                c = (x.end - x.begin) * tile_units(w, v, item_at(k0 + lane, items)) + w.start;
            }
            const int64_t sum = warp_scan(c);
            const unsigned in = __ballot_sync(0xffffffffu, off < sum);
            if (in != 0) {
                const int i = __ffs(in) - 1;
                off -= __shfl_sync(0xffffffffu, sum - c, i);
                k = k0 + i;
                break;
            }
            off -= __shfl_sync(0xffffffffu, sum, 31);
        }
        open(w);
        if (off == 0)
            return 0;
        const int tiles = begin_in(off, w.start);
        tile = t.begin + tiles;
        return static_cast<int>(w.start + static_cast<int64_t>(tiles) * units - off);
    }

    // Tiles that begin in n units from here, the first `ahead` of which begin none
    // but the one that stands here.
    __device__ __forceinline__ int begin_in(int64_t n, int ahead) const
    {
        return static_cast<int>(max((n - ahead + units - 1) / units, static_cast<int64_t>(1)));
    }

    // Tiles of the item that begin in the `left` (> 0) units of the run, and the
    // units that n of them take.
    __device__ __forceinline__ int run_tiles(const Work &w, int64_t left) const
    {
        return min(begin_in(left, tile == t.begin ? w.start : 0), t.end - tile);
    }
    __device__ __forceinline__ int64_t run_units(const Work &w, int n) const
    {
        return static_cast<int64_t>(n) * units + (tile == t.begin ? w.start : 0);
    }
};

// n / d where both mostly fit 32 bits, which divide several times faster.
__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d)
{
    return (n | d) >> 31 == 0 ? static_cast<uint32_t>(n) / static_cast<uint32_t>(d) : n / d;
}

// Deals the launch's units: those that worker `worker` has from the first tile
// that begins in its run, where `cur` is set (none: 0). A run is never shorter
// than a tile and an item's start, so that an item's parts lie in successive
// workers. Every warp of the block calls it (`workers` workers in all); `sums` is
// shared memory for MAX_GROUPS numbers that must not be used for anything else until
// the block has met again. Up to 32 sequences every warp counts by itself, without
// a barrier.
template <int BN>
__device__ __forceinline__ int64_t deal(const Work &w, int worker, int workers, int64_t *sums,
                                        Cursor<BN> &cur)
{
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int groups = (w.seqs.seqs + 31) / 32;
    int64_t n = 0, per_head = 0;
    if (groups == 1) {
        n = seq_units<BN>(w, 0);
        per_head = warp_sum(n);
    } else {
        for (int g = warp; g < groups; g += warps) {
            const int64_t x = warp_sum(seq_units<BN>(w, g));
            if ((threadIdx.x & 31) == 0)
                sums[g] = x;
        }
        __syncthreads();
        for (int g = threadIdx.x & 31; g < groups; g += 32)
            per_head += sums[g];
        per_head = warp_sum(per_head);
    }
    const int64_t units = per_head * w.kv_heads;
    const int shortest = w.full + w.start;
    if (workers > units / shortest)
        workers = static_cast<int>(max(units / shortest, static_cast<int64_t>(1)));
    if (worker >= workers)
        return 0;
    const int64_t base = quotient(units, workers);
    const int extra = static_cast<int>(units - base * workers);
    int64_t count = base + (worker < extra ? 1 : 0);
    if (count > 0) {
        const int64_t u = worker * base + min(worker, extra);
        cur.h = static_cast<int>(quotient(u, per_head));
        int64_t off = u - cur.h * per_head;
        int g = 0;
        if (groups > 1) {
            while (off >= sums[g])
                off -= sums[g++];
            n = seq_units<BN>(w, g);
        }
        count -= cur.seek(w, g, n, off);
        if (count > 0 && cur.tile == cur.t.end)
            cur.next_item(w);
    }
    return max(count, static_cast<int64_t>(0));
}

// Unnormalised sums of item parts, one slot per end of a worker's run:
// slot 2w holds the part of an item that began before worker w's run, slot
// 2w + 1 that of an item that begins in it and goes on behind it. The headers
// are written by every worker of every launch, so the workspace needs no
// initialisation.
struct PartHeader {
    int rows;              // of the item; 0: the slot is empty
    int more;              // 1: the item goes on in the next worker's first slot
    int row;               // first query row of the item's sequence
    int hm;                // key head + kv_heads * item number
};

struct Parts {
    PartHeader *headers;   // [2 * workers]
    float2 *ml;            // [2 * workers][row_cap]: maximum (log2 units) and sum
    float *o;              // [2 * workers]: [row_cap][head_dim], or with flags
                           // [head_dim / 4][row_cap][4], which a thread per row
                           // writes and reads in whole lines
    uint64_t *flags;       // [workers][16] or null: see the chunk kernel's output
    int row_cap;
};

}  // namespace paged
}  // namespace bitlinear
