// What the operators on the paged key/value cache share: the step's sequences
// as the device sees them, with every index from device memory checked before
// it is used, and the division of the attention's work between workers.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace bitlinear {
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

// Sequence s, cut to the rows and the page slots that exist (a value outside
// them is recorded as a fault).
__device__ __forceinline__ View view(const Seqs &q, int s)
{
    const int b = __ldg(q.q_start + s), e = __ldg(q.q_start + s + 1), n = __ldg(q.kv_len + s);
    View v;
    v.q0 = min(max(b, 0), q.tokens);
    v.qlen = min(max(e, v.q0), q.tokens) - v.q0;
    v.kv = min(max(n, 0), q.table_cols << q.page_shift);
    if (v.q0 != b || v.q0 + v.qlen != e || v.kv != n)
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
// The attention's work is cut into items: BM consecutive rows of one sequence
// and key head, where row r is query head r % group of token r / group, so the
// query heads that share a key head share its tiles. An item takes one unit
// per tile of BN keys that any of its rows sees. All units of a launch, items
// in order and key heads outermost, are dealt to the workers in equal
// contiguous runs: a long sequence is split wherever a run ends, and a batch
// of ragged ones stays balanced without the host knowing a length. A worker
// that gets a whole item writes its output; otherwise it leaves a partial sum
// that the merge kernel joins in the order of the keys.

struct Work {
    Seqs seqs;
    int group;             // query heads per key head
    int kv_heads;
    int window;            // 0: none
    int min_rows, max_rows;  // sequences of this launch: min_rows <= qlen * group <= max_rows
};

constexpr int MAX_GROUPS = 512;          // of 32 sequences: at most 16384 sequences

struct Tiles {
    int begin, end;        // key tiles
    int klo, khi;          // keys that any row of the item sees
};

template <int BM, int BN>
__device__ __forceinline__ Tiles item_tiles(const Work &w, const View &v, int m)
{
    const int r1 = min((m + 1) * BM, v.qlen * w.group) - 1;
    const int first = v.kv - v.qlen + (m * BM) / w.group;   // position of the first row
    const int last = v.kv - v.qlen + r1 / w.group;
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

template <int BM, int BN>
__device__ __forceinline__ int64_t seq_units(const Work &w, int s)
{
    if (s >= w.seqs.seqs)
        return 0;
    const View v = view(w.seqs, s);
    if (!in_launch(w, v))
        return 0;
    int64_t n = 0;
    for (int m = 0; m * BM < v.qlen * w.group; ++m) {
        const Tiles t = item_tiles<BM, BN>(w, v, m);
        n += t.end - t.begin;
    }
    return n;
}

// Units of every group of 32 sequences into sums[] (shared memory). Every warp
// of the block calls it; a block barrier follows.
template <int BM, int BN>
__device__ __forceinline__ void group_units(const Work &w, int warp, int warps, int64_t *sums)
{
    const int lane = threadIdx.x & 31;
    const int groups = (w.seqs.seqs + 31) / 32;
    for (int g = warp; g < groups; g += warps) {
        int64_t n = seq_units<BM, BN>(w, g * 32 + lane);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            n += __shfl_xor_sync(0xffffffffu, n, o);
        if (lane == 0)
            sums[g] = n;
    }
}

// A position in the launch's units: the item and the tile inside it.
template <int BM, int BN>
struct Cursor {
    int h, s, m, tile;
    View v;
    Tiles t;

    __device__ __forceinline__ void open(const Work &w)
    {
        t = item_tiles<BM, BN>(w, v, m);
        tile = t.begin;
    }

    // The first unit of the next item. Only called while units are left, so a
    // sequence of this launch is always found.
    __device__ __forceinline__ void next_item(const Work &w)
    {
        if (++m * BM >= v.qlen * w.group) {
            m = 0;
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

    // Moves to unit u of a launch of `per_head` units a key head (the whole
    // warp, with the block's group sums).
    __device__ __forceinline__ void seek(const Work &w, const int64_t *sums, int64_t per_head,
                                         int64_t u)
    {
        const int lane = threadIdx.x & 31;
        h = static_cast<int>(u / per_head);
        int64_t off = u - h * per_head;
        int g = 0;
        while (off >= sums[g])
            off -= sums[g++];
        const int64_t n = seq_units<BM, BN>(w, g * 32 + lane);
        int64_t upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o)
                upto += x;
        }
        const int at = __ffs(__ballot_sync(0xffffffffu, off < upto)) - 1;
        off -= __shfl_sync(0xffffffffu, upto - n, at);
        s = g * 32 + at;
        v = view(w.seqs, s);
        m = 0;
        open(w);
        while (off >= t.end - t.begin) {
            off -= t.end - t.begin;
            ++m;
            open(w);
        }
        tile = t.begin + static_cast<int>(off);
    }
};

// Unnormalised sums of item parts, one slot per end of a worker's run:
// slot 2w holds the part of an item that began before worker w's run, slot
// 2w + 1 that of an item that begins in it and goes on behind it. The headers
// are written by every worker of every launch, so the workspace needs no
// initialisation.
struct PartHeader {
    int state;             // 0: empty, 1: more parts follow, 2: the item's last part
    int s, m, h;
};

struct Parts {
    PartHeader *headers;   // [2 * workers]
    float2 *ml;            // [2 * workers][row_cap]: maximum (log2 units) and sum
    float *o;              // [2 * workers][row_cap][head_dim]
    int row_cap;
};

}  // namespace paged
}  // namespace bitlinear
