// Attention of many query rows over a paged cache (chunks of prompts and whole
// prompts) on the fifth-generation tensor cores.
//
// An item is up to 256 rows of one sequence and key head in two halves of at
// most 128, as many whole tokens as fit (a token is the group's query heads), so
// that a half's queries are one box of a tensor map; each half is a tcgen05.mma
// of M = 128. Per step of 64 keys and half h:
//   S_h = Q_h K^T          both operands from shared memory, S_h in TMEM
//   P_h = 2^(scale S_h - m) by eight warps, bf16 back into the columns of S_h
//   O_h += P_h V           P_h from TMEM, V from shared memory as it lies there
//                          (its channels contiguous: an MN-major operand)
// Each half has two S buffers, which the two steps of a 128-key tile take in
// turn: the products of one step run while the warps compute the exponentials of
// the other. A row's 64 scores of a step belong to two threads of two warps,
// which exchange their maxima through shared memory.
//
// What bounds it at D = 128: a tile of both halves takes 3700 to 3900 clocks (2.2
// us), against 2048 of the tensor pipe at its full rate. Products of N = 64 cost
// the pipe nearly what those of N = 128 do, so the scores take 2048 of these
// clocks instead of 1024, and the warps' chain of load, maximum, exponentials and
// store the rest. Measured beside it: one S buffer of 128 keys a half with one
// issuing warp 4580 clocks, with two issuing warps and two threads a row 4400;
// eight softmax warps with a row a thread 4000 (the same time where the clock is
// held down by power, but 20% slower on windowed prompts of 64 channels); every
// pair of exponentials on the special-function unit 4% slower, every second on
// the multiply-add pipe 4% slower. 4096 rows behind 28672 keys, 64 heads on 8:
// 4.0 to 4.5 ms, 920 to 1030 TFLOP/s, in calls back to back, by the clock that power
// leaves (3.7 ms on its own).
//
// Items that are split into up to four parts, as most split ones are, are joined
// here: a worker computes the part of the item that began before its run first
// and raises a flag per warp behind it; the item's first worker comes to its
// part last, finds the flags of the same warp (same rows, same channels) and
// adds the parts to its own, in the order of the keys, before it writes the
// output. The flags hold the launch's number, so their memory needs no
// initialisation; the kernel behind this one, which joins items of more parts,
// clears them. Runs are numbered from the last block to the first, so that a block
// waits only for blocks of a lower number. The GPU starts blocks in the order of
// their numbers: what is waited for runs already or is done, however few SMs other
// work leaves to the launch. (The other numbering, in which the waiting blocks start
// first, is 0.5 us of 46 faster at 2048 tokens of the 2B layer. Leaving every part to a
// kernel of its own took 18 us of 60 there.)
//
// One persistent block per SM. Warps 0-7 and 8-15 compute the halves' softmax,
// warp 16 fetches keys and values through a ring of tiles, and the next item's
// queries as soon as the last scores of this one are done, warps 17 and 18 issue the
// products of one half each. (A warp of its own for the queries made the compiler
// spill 156 bytes instead of 8: a 2048-token prompt 46.9 us instead of 44.7.) A warp
// whose row's maximum has grown rescales its rows of O_h itself, after the products
// of the previous step (its o_done).
#pragma once

#include "attn_rows.cuh"
#include "f32x2.cuh"

namespace bitlinear {
namespace attn {
namespace chunk {

constexpr int HALF = 128;              // most rows of a half item
constexpr int BN = 128;                // keys of a tile
constexpr int STEP = 64;               // keys of a step: the tile's two halves
constexpr int SOFTMAX_WARPS = 16;
constexpr int THREADS = (SOFTMAX_WARPS + 3) * 32;
constexpr int TMEM_COLS = 512;
constexpr int JOIN = 3;                // parts behind its own that a worker joins

// The worker (the run of units) of a block. Workers wait for the JOIN next ones.
__host__ __device__ constexpr int worker_of(int block, int blocks) { return blocks - 1 - block; }

// Limit of a wait for another worker's part. Runs are equal and the other one's block
// started no later, but its SM may be slower (it shares it with other work), so it is
// late by a part of the run's own time, which has no limit: `base_ns`, as for the waits
// inside a block, and ten times the 0.45 us that a unit takes, up to a minute.
// `units`: an upper bound of a run's.
__host__ __device__ constexpr uint64_t join_wait_ns(uint64_t base_ns, double units)
{
    return base_ns + static_cast<uint64_t>(units < 60e9 / 4500.0 ? units * 4500.0 : 60e9);
}

__device__ __forceinline__ uint64_t ld_acquire_u64(const uint64_t *p)
{
    uint64_t v;
    asm volatile("ld.acquire.gpu.global.b64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void st_release_u64(uint64_t *p, uint64_t v)
{
    asm volatile("st.release.gpu.global.b64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}

// Waits until the flag is nonce or nonce + 1 and returns it; 0 after the limit,
// or when the block gives up.
__device__ __forceinline__ uint64_t wait_flag(const uint64_t *flag, uint64_t nonce,
                                              volatile int *abort, uint64_t limit_ns)
{
    const uint64_t t0 = global_timer_ns();
    for (uint32_t spin = 0;; ++spin) {
        const uint64_t v = ld_acquire_u64(flag);
        if ((v & ~uint64_t(1)) == nonce)
            return v;
        if ((spin & 63u) == 63u) {
            if (*abort)
                return 0;
            if (global_timer_ns() - t0 > limit_ns) {
                atomicOr(&g_fault_word, FAULT_WAIT_TIMEOUT);
                *abort = 1;
                return 0;
            }
        }
    }
}

template <int D>
struct Cfg {
    static constexpr int CH = D / 64;                          // 64-channel column blocks
    static constexpr int Q_BYTES = HALF * D * 2;               // one half
    static constexpr int TILE_BYTES = BN * D * 2;              // keys or values of a tile
    static constexpr int STAGES = D == 128 ? 4 : 8;
    static constexpr int OUT_BYTES = 32 * 64;                  // staged output of one warp
    static constexpr int BARRIERS = 2 * STAGES + 19;
    // shared memory, all of it dynamic: queries, ring, the warps' staging,
    // barriers, TMEM address and abort flag
    static constexpr int RING_AT = 2 * Q_BYTES;
    static constexpr int OUT_AT = RING_AT + STAGES * TILE_BYTES;
    static constexpr int BAR_AT = OUT_AT + SOFTMAX_WARPS * OUT_BYTES;
    static constexpr int SMEM_BYTES = BAR_AT + BARRIERS * 8 + 16;
};

// True in one lane of the warp. A branch on it (rather than on a lane number)
// tells the compiler that a single lane runs the issuing code, so that the
// descriptors go straight to the uniform registers that the instructions take
// them from.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, e;\n\t}"
        : "=r"(r));
    return r != 0;
}

// D[tmem] (+)= A[smem] B[smem]^T, bf16 inputs, fp32 accumulator.
__device__ __forceinline__ void umma_bf16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The same with A in TMEM: lane = row, two bf16 per column, k = 16 in 8 columns.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                             uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor: kind::f16, bf16 x bf16 -> fp32, A K-major, B K-major
// or MN-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n, bool b_mn_major)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn_major ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// Descriptor of an MN-major operand in the 128-byte swizzled layout: 64
// channels (128 bytes) by 8 keys are one 1024-byte atom, the next 8 keys
// follow it (stride offset), the next 64 channels lie `ch_bytes` further
// (leading offset).
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t ch_bytes)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(ch_bytes >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// Ties 32 registers of a TMEM load to what was waited for before it: their
// readers cannot be moved in front.
__device__ __forceinline__ void loaded32(uint32_t *r)
{
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                   "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31]));
}

// 2^x of two lanes on the multiply-add pipe, for -126 <= x < 127: x = n + f with
// n the nearest integer (the low bits of x + 1.5 * 2^23), 2^f by the degree-4
// polynomial of least relative error on [-1/2, 1/2] (2.7e-6, Remez exchange),
// n added to its exponent. The special-function unit gives 16 results a clock
// and SM and would bound the kernel alone; every fourth pair goes this way.
__device__ __forceinline__ void exp2_poly2(uint64_t x, float &lo, float &hi)
{
    float a, b;
    unpair(x, a, b);
    x = pair(fmaxf(a, -126.0f), fmaxf(b, -126.0f));
    const uint64_t r = add2(x, pair(12582912.0f, 12582912.0f));
    const uint64_t n = add2(r, pair(-12582912.0f, -12582912.0f));
    const uint64_t f = fma2(n, pair(-1.0f, -1.0f), x);
    uint64_t q = fma2(pair(0.009570102207362652f, 0.009570102207362652f), f,
                      pair(0.05591785907745361f, 0.05591785907745361f));
    q = fma2(q, f, pair(0.240247443318367f, 0.240247443318367f));
    q = fma2(q, f, pair(0.6931217908859253f, 0.6931217908859253f));
    q = fma2(q, f, pair(0.9999992847442627f, 0.9999992847442627f));
    float n0, n1;
    unpair(r, n0, n1);
    unpair(q, lo, hi);
    lo = __uint_as_float(__float_as_uint(lo) + (__float_as_uint(n0) << 23));
    hi = __uint_as_float(__float_as_uint(hi) + (__float_as_uint(n1) << 23));
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 16 columns of the warp's 32 lanes, waited for.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    attn_chunk_kernel(const __grid_constant__ Maps maps, const __grid_constant__ CUtensorMap q_map,
                      const Params p)
{
    using C = Cfg<D>;
    using Cursor = paged::Cursor<BN>;

    // The swizzled tiles start on 1024-byte boundaries: the kernel has no other
    // shared memory, so the array begins where the block's does.
    extern __shared__ __align__(1024) char smem[];
    const int lane = threadIdx.x & 31;
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const uint32_t smem0 = smem_u32(smem);
    const uint32_t q_smem = smem0;                             // [half][column block][row][128 B]
    const uint32_t ring = smem0 + C::RING_AT;                  // [stage][column block][key][128 B]
    int64_t *sums = reinterpret_cast<int64_t *>(smem);         // while the work is dealt
    volatile uint32_t *tmem_slot =
        reinterpret_cast<volatile uint32_t *>(smem + C::BAR_AT + C::BARRIERS * 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    auto bar = [&](int i) { return smem0 + C::BAR_AT + i * 8; };
    auto full = [&](int s) { return bar(s); };
    auto empty = [&](int s) { return bar(C::STAGES + s); };
    auto q_ready = [&](int h) { return bar(2 * C::STAGES + h); };
    auto o_done = [&](int h, int b) { return bar(2 * C::STAGES + 2 + 2 * h + b); };
    auto s_full = [&](int h, int b) { return bar(2 * C::STAGES + 6 + 2 * h + b); };
    auto p_ready = [&](int h, int b) { return bar(2 * C::STAGES + 10 + 2 * h + b); };
    auto drain_bar = [&](int h) { return bar(2 * C::STAGES + 14 + h); };
    auto q_free = [&](int h) { return bar(2 * C::STAGES + 16 + h); };
    const uint32_t part_done = bar(2 * C::STAGES + 18);        // the first item's, by every warp

    if (threadIdx.x == 0) {
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
        prefetch_tensormap(&q_map);
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full(s), 1 + (s == 0 && worker_of(blockIdx.x, gridDim.x) == p.stuck));
            mbar_init(empty(s), 2);                            // both halves
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(q_ready(h), 1);
            mbar_init(q_free(h), 1);
            mbar_init(drain_bar(h), 1);
            for (int b = 0; b < 2; ++b) {
                mbar_init(o_done(h, b), 1);
                mbar_init(s_full(h, b), 1);
                mbar_init(p_ready(h, b), 8);
            }
        }
        mbar_init(part_done, SOFTMAX_WARPS);
        fence_barrier_init();
        *abort_flag = 0;
    }
    if (warp == 17)
        tmem_alloc(smem0 + C::BAR_AT + C::BARRIERS * 8, TMEM_COLS);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();
    const paged::Work &w = p.work;
    const int worker = worker_of(blockIdx.x, gridDim.x);
    Cursor cur;
    const int64_t count = paged::deal<BN>(w, worker, gridDim.x, sums, cur);
    if (w.seqs.seqs > 32) {
        // sums is read; its memory is Q's, which TMA writes: a barrier alone does not
        // order these accesses before those of the other proxy
        fence_proxy_async();
        __syncthreads();
    }

    // The whole warp waits; false after a timeout anywhere in the block.
    auto wait = [&](uint32_t b, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_try_wait(b, parity)) ||
               warp_wait_bounded(b, parity, abort_flag, p.wait_limit_ns);
    };
    // S buffer b of half h at column h * 128 + b * 64 (P in its first 32), O_h
    // behind them.
    auto s_tmem = [&](int h, int b) { return tmem + h * 128 + b * STEP; };
    auto o_tmem = [&](int h) { return tmem + 256 + h * 128; };
    const int half_rows = w.item_rows / 2;                     // whole tokens, at most HALF rows
    auto rows_of = [&]() { return min(w.item_rows, cur.v.qlen * w.group - cur.m * w.item_rows); };
    auto halves_of = [&]() { return rows_of() > half_rows ? 2 : 1; };

    // Whether no row of the item sees the first, or the last, step of its tiles in
    // this run. Such a step passes its barriers, but nothing is computed; one step
    // of an item is always left. Only with 64 channels, where windowed prompts take
    // 205 us instead of 218: with 128 the code spills 144 bytes more and a 2048-token
    // prompt takes 47.2 us instead of 44.6.
    constexpr bool SKIP = D == 64;
    auto unseen_first = [&]() { return SKIP && cur.tile * BN + STEP <= cur.t.klo; };
    auto unseen_last = [&](int nt) {
        return SKIP && (cur.tile + nt) * BN - STEP >= cur.t.khi;
    };

    // element of channel 0 of row i of cursor c's item in a tensor of rows
    auto row_of = [&](const Cursor &c, int i, int64_t stride) {
        const int rr = c.m * w.item_rows + i;
        const int tok = w.by_group(rr);
        return (c.v.q0 + tok) * stride + (c.h * w.group + rr - tok * w.group) * D;
    };

    paged::PartHeader head[2] = {};
    int64_t left = count;
    if (warp == 16) {
        // ======================================= queries, keys and values
        // An item's queries come between its first keys and the values beside
        // them: their place is free once the last scores of the item before are
        // done, when those keys are under way. A box is whole tokens and the group's
        // heads: its rows are the half's. Rows behind the sequence's last come along
        // (those of other tokens, or zeros); whatever they hold stays in rows that
        // are never stored.
        //
        // This warp also raises the flags behind a part that another worker joins
        // (the run's first item, if that began in an earlier run): the fence ahead
        // of them waits two microseconds for the part's stores, which would hold
        // the softmax warps back. It does so when two tiles of the next item are in
        // the ring.
        const int page = 1 << w.seqs.page_shift;
        const int box = min(page, BN), subs = BN / box, boxes = subs * C::CH;
        int st = 0;
        uint32_t ph = 0, armed = 0;                            // armed: stages in flight, as bits
        uint32_t q_ph[2] = {0, 0};
        int fetched[2] = {0, 0};
        uint64_t flag = 0;
        bool ok = true;
        auto raise_flags = [&]() {
            ok = wait(part_done, 0u);
            if (ok) {
                __threadfence();
                if (lane < SOFTMAX_WARPS)
                    st_release_u64(p.parts.flags + worker * SOFTMAX_WARPS + lane, flag);
            }
            flag = 0;
        };
        auto fetch_queries = [&]() {
            const int tok = cur.v.q0 + w.by_group(cur.m * w.item_rows);
            for (int h = 0; ok && h < halves_of(); ++h) {
                ok = wait(q_free(h), q_ph[h] ^ 1u);
                if (!ok)
                    break;
                q_ph[h] ^= 1u;
                fetched[h] = 1;
                if (elect_one()) {
                    mbar_arrive_expect_tx(q_ready(h), half_rows * D * 2);
                    for (int c = 0; c < C::CH; ++c)
                        tma_load_3d(q_smem + h * C::Q_BYTES + c * (HALF * 128), &q_map, c * 64,
                                    cur.h * w.group, tok + h * w.by_group(half_rows),
                                    q_ready(h));
                }
                __syncwarp();
            }
        };
        while (ok && left > 0) {
            const int nt = cur.run_tiles(w, left);
            const bool due = flag != 0;                        // behind the item before
            if (cur.tile != cur.t.begin)
                flag = p.nonce + (cur.tile + nt == cur.t.end ? 0 : 1);
            for (int j = 0; ok && j < nt; ++j) {
                if (j == 2 && due) {
                    raise_flags();
                    if (!ok)
                        break;
                }
                const int sub = lane % subs, ch = (lane / subs) % C::CH;
                const int key = (cur.tile + j) * BN + sub * box;
                // a box without a needed key, or of a page that the table does
                // not hold, starts behind the cache and is filled with zeros
                int row = p.cache_rows;
                if (lane < boxes && key < cur.t.khi && key + box > cur.t.klo) {
                    const int id = paged::page_of(w.seqs, cur.s, key >> w.seqs.page_shift);
                    if (id >= 0)
                        row = ((id * w.kv_heads + cur.h) << w.seqs.page_shift) + (key & (page - 1));
                }
                for (int kv = 0; ok && kv < 2; ++kv) {
                    if (!wait(empty(st), ph ^ 1u)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0)
                        mbar_arrive_expect_tx(full(st), C::TILE_BYTES);
                    __syncwarp();
                    if (lane < boxes)
                        tma_load_2d(ring + st * C::TILE_BYTES + ch * (BN * 128) + sub * box * 128,
                                    kv == 0 ? &maps.k : &maps.v, ch * 64, row, full(st));
                    armed |= 1u << st;
                    if (++st == C::STAGES) {
                        st = 0;
                        ph ^= 1u;
                    }
                    if (j == 0 && kv == 0)
                        fetch_queries();
                }
            }
            if (ok && due && flag != 0)
                raise_flags();
            left -= cur.run_units(w, nt);
            if (ok && left > 0)
                cur.next_item(w);
        }
        if (ok && flag != 0)
            raise_flags();
        // No copy is left in flight when the block ends, whichever of its warps gave up
        // (this one may be done when another does): a stage's last phase is the one
        // before its next fill.
        if (lane == 0) {
            for (int s = 0; s < C::STAGES; ++s)
                if ((armed >> s) & 1u)
                    drain_wait(full(s), s < st ? ph : ph ^ 1u, p.wait_limit_ns);
            for (int h = 0; h < 2; ++h)
                if (fetched[h])
                    drain_wait(q_ready(h), q_ph[h] ^ 1u, p.wait_limit_ns);
        }
        __syncwarp();
    } else if (warp == 17 || warp == 18) {
        // ============================================== products of half h
        constexpr uint32_t S_IDESC = idesc_bf16(HALF, STEP, false);
        constexpr uint32_t O_IDESC = idesc_bf16(HALF, D, true);
        constexpr uint32_t STEP_OFF = STEP * 128 / 16;         // 64 keys further, in 16 bytes
        const int h = warp - 17;
        const uint64_t q_desc = smem_desc_k128_sw128(q_smem + h * C::Q_BYTES);
        const uint64_t k_desc = smem_desc_k128_sw128(ring);
        const uint64_t v_desc = smem_desc_mn_sw128(ring, BN * 128);
        int st = 0;
        uint32_t ph = 0, q_ph = 0, p_ph = 0;
        bool ok = true;
        auto next_stage = [&]() {
            if (++st == C::STAGES) {
                st = 0;
                ph ^= 1u;
            }
        };
        auto scores = [&](int b, int stage, bool unseen) {
            const uint64_t k = k_desc + stage * (C::TILE_BYTES / 16) + b * STEP_OFF;
            if (!unseen) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    // 16 channels are 32 bytes of a 128-byte row, 64 a column block
                    const uint64_t off = (i >> 2) * (HALF * 128 / 16) + (i & 3) * 2;
                    umma_bf16_ss(s_tmem(h, b), q_desc + off, k + off, S_IDESC, i > 0);
                }
            }
            umma_commit(s_full(h, b));
        };
        while (ok && left > 0) {
            const int nt = cur.run_tiles(w, left);
            if (h < halves_of()) {
                const bool first_unseen = unseen_first(), last_unseen = unseen_last(nt);
                int k_stage = st;
                ok = wait(q_ready(h), q_ph) && wait(full(st), ph);
                q_ph ^= 1u;
                if (!ok)
                    break;
                next_stage();
                tc_fence_after_sync();
                if (elect_one()) {
                    scores(0, k_stage, first_unseen);
                    scores(1, k_stage, nt == 1 && last_unseen);
                    umma_commit(empty(k_stage));
                    if (nt == 1)
                        umma_commit(q_free(h));
                }
                __syncwarp();
                for (int j = 0; j < nt; ++j) {
                    const int v_stage = st;
                    ok = wait(full(st), ph);
                    if (!ok)
                        break;
                    next_stage();
                    const int key0 = (cur.tile + j) * BN;
                    const int skip = max(cur.t.klo - key0, 0), upto = min(cur.t.khi - key0, BN);
                    if (skip > 0 || upto < BN) {
                        // slots that hold no key of the sequence may hold
                        // anything, and 0 * NaN is NaN: their values become
                        // zeros (the halves' warps write the same ones)
                        for (int i = lane; i < BN * 8 * C::CH; i += 32) {
                            const int key = (i >> 3) & (BN - 1);
                            if (key < skip || key >= upto)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                                 ring + v_stage * C::TILE_BYTES + i * 16),
                                             "r"(0)
                                             : "memory");
                        }
                        fence_proxy_async();
                        __syncwarp();
                    }
                    const bool more = j + 1 < nt;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        ok = ok && wait(p_ready(h, b), p_ph);
                        if (!ok)
                            break;
                        tc_fence_after_sync();
                        const bool unseen =
                            b == 0 ? j == 0 && first_unseen : j + 1 == nt && last_unseen;
                        if (elect_one()) {
                            const uint64_t v =
                                v_desc + v_stage * (C::TILE_BYTES / 16) + b * STEP_OFF;
                            if (!unseen) {
#pragma unroll
                                for (int i = 0; i < STEP / 16; ++i)    // 16 keys: two atoms
                                    umma_bf16_ts(o_tmem(h), s_tmem(h, b) + i * 8,
                                                 v + i * (2048 / 16), O_IDESC,
                                                 j > 0 || (b > 0 && !first_unseen) || i > 0);
                            }
                            umma_commit(o_done(h, b));
                            if (b == 1)
                                umma_commit(empty(v_stage));
                        }
                        __syncwarp();
                        if (more) {
                            if (b == 0) {
                                k_stage = st;
                                ok = wait(full(st), ph);
                                if (!ok)
                                    break;
                                next_stage();
                            }
                            if (elect_one()) {
                                scores(b, k_stage, b == 1 && j + 2 == nt && last_unseen);
                                if (b == 1)
                                    umma_commit(empty(k_stage));
                                if (b == 1 && j + 2 == nt)
                                    umma_commit(q_free(h));
                            }
                            __syncwarp();
                        }
                    }
                    p_ph ^= 1u;
                    if (!ok)
                        break;
                }
            } else {
                // the item has no rows in this half: give its tiles back
                for (int j = 0; ok && j < 2 * nt; ++j) {
                    ok = wait(full(st), ph);
                    if (ok && lane == 0)
                        mbar_arrive(empty(st));
                    next_stage();
                }
            }
            left -= cur.run_units(w, nt);
            if (ok && left > 0)
                cur.next_item(w);
        }
        if (elect_one()) {                                     // nothing in flight at the end
            umma_commit(drain_bar(h));
            drain_wait(drain_bar(h), 0u, p.wait_limit_ns);
        }
        __syncwarp();
    } else {
        // ======================================================== softmax
        const int h = warp >> 3;                               // half of the item
        const int part = (warp >> 2) & 1;                      // 32 of the step's 64 keys
        const int in_half = (warp & 3) * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_addr = s_tmem(h, 0) + lane_off + part * 32;
        const uint32_t p_addr = s_tmem(h, 0) + lane_off + part * 16;
        const uint32_t o_addr = o_tmem(h) + lane_off + part * (D / 2);
        char *out = smem + C::OUT_AT + warp * C::OUT_BYTES;
        const int pair_bar = 1 + h * 4 + (warp & 3);           // the two warps of 32 rows
        const char *other = smem + C::OUT_AT + (warp ^ 4) * C::OUT_BYTES;
        // A row's other thread finds its maximum (of two steps in turn) and sum in
        // this warp's staging rows, which hold output only between the items'
        // last barrier and the next one's first maximum.
        float *const my_max = reinterpret_cast<float *>(out) + lane;
        const float *const other_max = reinterpret_cast<const float *>(other) + lane;
        uint32_t ph = 0;                                       // parity of the tile's barriers
        bool ok = true;
        while (ok && left > 0) {
            const int nt = cur.run_tiles(w, left);
            const bool from_start = cur.tile == cur.t.begin;
            const bool to_end = cur.tile + nt == cur.t.end;
            const int rows = rows_of();
            const int slot = 2 * worker + (from_start ? 1 : 0);
            const bool whole = from_start && to_end;
            const bool active = h < halves_of();
            if (!whole)
                head[from_start ? 1 : 0] =
                    paged::PartHeader{rows, to_end ? 0 : 1, cur.v.q0, cur.h + w.kv_heads * cur.m};
            // this thread's row of the item, and those of its half
            const int r = h * half_rows + in_half;
            const int end = min(rows, (h + 1) * half_rows);
            const int rr = cur.m * w.item_rows + r;
            const int tok = w.by_group(rr);
            // a warp without a row leaves its lanes of P as they are: they only
            // reach rows of O that nobody reads
            const bool idle = r - lane >= end;
            float m = -INFINITY, l = 0.0f;
            if (active) {
                const int seen_hi = cur.v.kv - cur.v.qlen + tok;     // last key the row sees
                // keys that every row of this warp sees: steps inside need no mask
                const int all_hi = __shfl_sync(0xffffffffu, seen_hi, 0);
                const int all_lo =
                    w.window > 0 ? __shfl_sync(0xffffffffu, seen_hi, 31) - w.window + 1 : 0;
                const int first = unseen_first() ? 1 : 0;
                const int steps = 2 * nt - (unseen_last(nt) ? 1 : 0);
                if (first > 0) {
                    ok = ok && wait(s_full(h, 0), ph);
                    if (ok && lane == 0)
                        mbar_arrive(p_ready(h, 0));
                }
                for (int j = first; j < steps; ++j) {
                    const int b = j & 1;
                    ok = ok && wait(s_full(h, b), ph);
                    if (idle) {                                // no row to compute
                        if (!ok)
                            break;
                        ph ^= static_cast<uint32_t>(b);
                        if (lane == 0)
                            mbar_arrive(p_ready(h, b));
                        continue;
                    }
                    tc_fence_after_sync();
                    uint32_t s[32];
                    tmem_ld_32x32b_x32(s_addr + b * STEP, s);
                    tmem_ld_wait();
                    loaded32(s);
                    const int key0 = cur.tile * BN + j * STEP;
                    const bool masked = key0 + STEP - 1 > all_hi || key0 < all_lo;
                    if (masked) {
                        const int hi = seen_hi - key0 - part * 32;
                        const int lo = w.window > 0 ? hi - w.window : -1;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i > hi || i <= lo)
                                s[i] = 0xff800000u;
                    }
                    float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            t4[k] = max3(__uint_as_float(s[i + 2 * k]),
                                         __uint_as_float(s[i + 2 * k + 1]), t4[k]);
                    // The row's maximum from both its threads. The barrier also
                    // takes the two warps' verdict on their waits, so that neither
                    // is left alone at the next one.
                    const float mine = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
                    my_max[b * 32] = mine;
                    ok = named_bar_and(pair_bar, 64, ok);
                    if (!ok)
                        break;
                    const float top = fmaxf(mine, other_max[b * 32]) * p.scale_log2;
                    const bool raise = top > m + RESCALE_AT;           // also from -inf
                    if (__any_sync(0xffffffffu, raise)) {
                        const float f = raise ? exp2_approx(m - top) : 1.0f;
                        if (raise)
                            m = top;
                        l *= f;
                        if (j > 0) {
                            // O_h rests after the last step's products (those of
                            // the step before went ahead of this step's scores);
                            // each of the two warps rescales half its channels
                            ok = wait(o_done(h, b ^ 1), b == 1 ? ph : ph ^ 1u);
                            tc_fence_after_sync();
#pragma unroll 1
                            for (int c = 0; ok && c < D / 32; ++c) {
                                uint32_t o[16];
                                tmem_ld_x16(o_addr + c * 16, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tmem_st_x16(o_addr + c * 16, o);
                            }
                        }
                    }
                    ph ^= static_cast<uint32_t>(b);
                    const float sub = m == -INFINITY ? 0.0f : m;
                    const uint64_t scale2 = pair(p.scale_log2, p.scale_log2);
                    const uint64_t sub2 = pair(-sub, -sub);
                    uint64_t sum[2] = {0, 0};
                    auto weights = [&](auto exact) {
                        uint32_t e[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const uint64_t x = fma2(
                                pair(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])),
                                scale2, sub2);
                            float a, b;
                            if (!decltype(exact)::value && i % 4 == 3) {
                                exp2_poly2(x, a, b);
                            } else {
                                unpair(x, a, b);
                                a = exp2_approx(a);
                                b = exp2_approx(b);
                            }
                            sum[i & 1] = add2(sum[i & 1], pair(a, b));
                            e[i] = pack_bf16(a, b);
                        }
                        tmem_st_x16(p_addr + b * STEP, e);
                    };
                    // a masked score is -inf and must weigh exactly nothing
                    if (masked)
                        weights(std::true_type{});
                    else
                        weights(std::false_type{});
                    tmem_st_wait();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(p_ready(h, b));
                    float a, c;
                    unpair(add2(sum[0], sum[1]), a, c);
                    l += a + c;
                }
                if (ok && steps < 2 * nt) {
                    ok = wait(s_full(h, 1), ph);
                    ph ^= 1u;
                    if (ok && lane == 0)
                        mbar_arrive(p_ready(h, 1));
                }
            }
            if (active) {
                // the last products; the row's sum from both its threads
                ok = ok && wait(o_done(h, 1), ph ^ 1u);
                if (!idle) {
                    // (the last products are done, so the other thread has read the
                    // maxima)
                    my_max[64] = l;
                    ok = named_bar_and(pair_bar, 64, ok);
                    l = part == 0 ? l + other_max[64] : other_max[64] + l;
                    ok = named_bar_and(pair_bar, 64, ok);      // both sums are read
                }
                if (!ok)
                    break;
                tc_fence_after_sync();
            }
            if (active && !idle) {
                const int64_t slot_row = static_cast<int64_t>(slot) * p.parts.row_cap + r;
                bool final = whole;
                float f = 1.0f, fk[JOIN];                      // factors of the parts
                int others = 0;                                // that are joined here
                const float4 *const o_parts =
                    reinterpret_cast<const float4 *>(p.parts.o) +
                    static_cast<int64_t>(part * (D / 8)) * p.parts.row_cap + r;
                const int64_t slot_o = static_cast<int64_t>(p.parts.row_cap) * (D / 4);
                if (from_start && !to_end) {
                    uint64_t flag = 0;
#pragma unroll
                    for (int k = 0; k < JOIN; ++k) {
                        if (final)
                            break;
                        if (lane == 0)
                            flag = wait_flag(p.parts.flags + (worker + 1 + k) * 16 + warp, p.nonce,
                                         abort_flag, p.join_limit_ns);
                        flag = __shfl_sync(0xffffffffu, flag, 0);
                        ok = named_bar_and(pair_bar, 64, flag != 0);
                        if (!ok)
                            break;
                        others = k + 1;
                        final = flag == p.nonce;               // this part ends the item
                    }
                    if (!ok)
                        break;
                    if (!final)
                        others = 0;                            // too many: left to the next kernel
                }
                if (others > 0) {
                    head[1].rows = 0;                          // nothing is left to merge
                    float2 ml[JOIN];
                    float top = m;
#pragma unroll
                    for (int k = 0; k < JOIN; ++k) {
                        ml[k] = make_float2(-INFINITY, 0.0f);
                        if (k < others && r < end)
                            ml[k] = __ldcg(p.parts.ml +
                                           static_cast<int64_t>(2 * (worker + 1 + k)) *
                                               p.parts.row_cap + r);
                        top = fmaxf(top, ml[k].x);
                    }
                    const float base = top == -INFINITY ? 0.0f : top;
                    f = exp2_approx(m - base);
                    l *= f;
                    m = top;
#pragma unroll
                    for (int k = 0; k < JOIN; ++k) {
                        fk[k] = exp2_approx(ml[k].x - base);
                        l = fmaf(ml[k].y, fk[k], l);
                    }
                }
                if (final) {
                    // This warp's half of the channels, 64 bytes of each row at a
                    // time through its staging rows, from where four lanes write a
                    // row's 64 bytes.
                    const float inv = inv_sum(l);
                    f *= inv;
                    char *dst[4];                              // of the rows that this lane writes
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = r - lane + i * 8 + (lane >> 2);
                        uint16_t *row = p.y + row_of(cur, at, p.y_stride) + part * (D / 2);
                        dst[i] = at < end ? reinterpret_cast<char *>(row) + (lane & 3) * 16
                                          : nullptr;
                    }
                    uint4 *const mine = reinterpret_cast<uint4 *>(out + lane * 64);
#pragma unroll 1
                    for (int c = 0; c < D / 64; ++c) {
                        uint32_t x[16], o[32];
                        tmem_ld_32x32b_x32(o_addr + c * 32, o);
                        tmem_ld_wait();
                        loaded32(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
#pragma unroll
                        for (int k = 0; k < JOIN; ++k) {
                            if (k >= others)
                                break;
                            const float4 *src = o_parts + 2 * (worker + 1 + k) * slot_o;
                            const float g = fk[k] * inv;
                            float4 v[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                v[i] = r < end ? __ldcg(src + (c * 8 + i) * p.parts.row_cap)
                                               : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float e[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    o[4 * i + q] = __float_as_uint(
                                        fmaf(e[q], g, __uint_as_float(o[4 * i + q])));
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            x[i] = pack_bf16(__uint_as_float(o[2 * i]),
                                             __uint_as_float(o[2 * i + 1]));
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mine[i ^ ((lane >> 1) & 3)] =
                                make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                        __syncwarp();
                        uint4 v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int at = i * 8 + (lane >> 2);        // row of the warp
                            v[i] = reinterpret_cast<const uint4 *>(
                                out + at * 64)[(lane & 3) ^ ((at >> 1) & 3)];
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (dst[i] != nullptr)
                                *reinterpret_cast<uint4 *>(dst[i] + c * 64) = v[i];
                        __syncwarp();
                    }
                    if (r < end && part == 0 && p.lse != nullptr)
                        p.lse[(cur.v.q0 + tok) * static_cast<int64_t>(p.q_heads) +
                              cur.h * w.group + rr - tok * w.group] = lse_of(m, l);
                } else {
                    float4 *mine = const_cast<float4 *>(o_parts) + slot * slot_o;
#pragma unroll 1
                    for (int c = 0; c < D / 64; ++c) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(o_addr + c * 32, o);
                        tmem_ld_wait();
                        loaded32(o);
                        if (r < end) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                mine[(c * 8 + i) * p.parts.row_cap] = make_float4(
                                    __uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                    __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                        }
                    }
                    if (r < end && part == 0)
                        p.parts.ml[slot_row] = make_float2(m, l);
                }
            }
            if (!from_start) {                                 // for the flags behind the part
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(part_done);
            }
            left -= cur.run_units(w, nt);
            if (left > 0)
                cur.next_item(w);
        }
        if (!ok)
            head[0].rows = head[1].rows = 0;                 // no part that could be merged
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 17) {
        tmem_relinquish();
        tmem_dealloc(tmem, TMEM_COLS);
    }
    if (threadIdx.x == 0) {
        if (*abort_flag)
            head[0].rows = head[1].rows = 0;
        p.parts.headers[2 * worker] = head[0];
        p.parts.headers[2 * worker + 1] = head[1];
    }
}

// Joins the items of more parts than that (one sequence's long context shared
// by many workers) and clears the flags. A warp takes 32 rows, one a lane, and
// four channels, of which every part is one whole line.
template <int D>
__global__ void __launch_bounds__(MERGE_THREADS) join_kernel(const MergeParams p)
{
    __shared__ paged::PartHeader begun[MERGE_WARPS];
    __shared__ int count[MERGE_WARPS];
    pdl_wait();
    pdl_launch_dependents();
    // (a captured launch raises the same flags every time it is replayed)
    for (int i = (blockIdx.y * gridDim.x + blockIdx.x) * MERGE_THREADS + threadIdx.x;
         i < 16 * p.workers; i += gridDim.x * gridDim.y * MERGE_THREADS)
        p.parts.flags[i] = 0;
    list_items(p, begun, count);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row_cap = p.parts.row_cap;
    for (int i = 0; i < MERGE_WARPS; ++i) {
        const int parts = count[i];
        if (parts == 0)
            continue;
        const paged::PartHeader hd = begun[i];
        const int first = 2 * (static_cast<int>(blockIdx.x) * MERGE_WARPS + i) + 1;
        const int m = hd.hm / p.work.kv_heads;
        const int units = (hd.rows + 31) / 32 * (D / 4);
        for (int u = blockIdx.y * MERGE_WARPS + warp; u < units; u += gridDim.y * MERGE_WARPS) {
            const int r = u / (D / 4) * 32 + lane, c4 = u % (D / 4);
            if (r >= hd.rows)
                continue;
            // part 0 is slot `first`, part k > 0 slot first + 2 k - 1
            auto slot = [&](int k) {
                return static_cast<int64_t>(first + (k > 0 ? 2 * k - 1 : 0)) * row_cap;
            };
            float top = -INFINITY;
#pragma unroll 8
            for (int k = 0; k < parts; ++k)
                top = fmaxf(top, p.parts.ml[slot(k) + r].x);
            const float base = top == -INFINITY ? 0.0f : top;
            float l = 0.0f;
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int k0 = 0; k0 < parts; k0 += 8) {
                float2 ml[8];
                float4 v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k0 + k < parts) {
                        ml[k] = p.parts.ml[slot(k0 + k) + r];
                        v[k] = reinterpret_cast<const float4 *>(p.parts.o)[
                            slot(k0 + k) * (D / 4) + static_cast<int64_t>(c4) * row_cap + r];
                    }
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k0 + k < parts) {
                        const float f = exp2_approx(ml[k].x - base);
                        l = fmaf(ml[k].y, f, l);
                        o.x = fmaf(v[k].x, f, o.x);
                        o.y = fmaf(v[k].y, f, o.y);
                        o.z = fmaf(v[k].z, f, o.z);
                        o.w = fmaf(v[k].w, f, o.w);
                    }
            }
            const int rr = m * p.work.item_rows + r;
            const int tok = p.work.by_group(rr);
            const int hq = (hd.hm - m * p.work.kv_heads) * p.work.group + rr - tok * p.work.group;
            const int64_t row = hd.row + tok;
            const float f = inv_sum(l);
            *reinterpret_cast<uint2 *>(p.y + row * p.y_stride + hq * D + 4 * c4) =
                make_uint2(pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f));
            if (p.lse != nullptr && c4 == 0)
                p.lse[row * p.q_heads + hq] = lse_of(top, l);
        }
    }
}

}  // namespace chunk
}  // namespace attn
}  // namespace bitlinear
