// Attention of many query rows over a paged cache (chunks of prompts and whole
// prompts) on the fifth-generation tensor cores.
//
// An item is 256 rows of one sequence and key head in two halves of 128, each
// a tcgen05.mma of M = 128. Per tile of 128 keys and half h:
//   S_h = Q_h K^T          both operands from shared memory, S_h in TMEM
//   P_h = 2^(scale S_h - m) by four warps, one row per thread, bf16 back into
//                          the columns of S_h
//   O_h += P_h V           P_h from TMEM, V from shared memory as it lies there
//                          (its channels contiguous: an MN-major operand)
// The products of one half run while the other half's warps compute its
// exponentials, which is what bounds the kernel: a tile takes 4 * 256 * 128 * D
// flops of the tensor pipe and 256 * 128 exponentials, about as many clocks of
// the special-function units at D = 128, and twice as many at D = 64.
//
// One persistent block per SM. Warps 0-3 and 4-7 compute the halves' softmax,
// warp 8 fetches keys and values through a ring of tiles, warp 9 issues the
// products. S_h(j + 1) is issued after P_h V_j, and a commit covers all
// products before it: a half's warps that see S_h(j + 1) know that O_h is at
// rest, so they rescale it themselves when their row's maximum has grown.
#pragma once

#include "attn_rows.cuh"

namespace bitlinear {
namespace attn {
namespace chunk {

constexpr int BM = 256, HALF = 128;    // rows of an item, of a half
constexpr int BN = 128;                // keys of a tile
constexpr int SOFTMAX_WARPS = 8;
constexpr int THREADS = (SOFTMAX_WARPS + 2) * 32;
constexpr int TMEM_COLS = 512;

template <int D>
struct Cfg {
    static constexpr int CH = D / 64;                          // 64-channel column blocks
    static constexpr int Q_BYTES = HALF * D * 2;               // one half
    static constexpr int TILE_BYTES = BN * D * 2;              // keys or values of a tile
    static constexpr int STAGES = D == 128 ? 5 : 8;
    static constexpr int SMEM_BYTES = 1024 + 2 * Q_BYTES + STAGES * TILE_BYTES;
};

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
    attn_chunk_kernel(const __grid_constant__ Maps maps, const Params p)
{
    using C = Cfg<D>;
    using Cursor = paged::Cursor<BM, BN>;

    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * C::STAGES + 9];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t smem0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t q_smem = smem0;                             // [half][column block][row][128 B]
    const uint32_t ring = smem0 + 2 * C::Q_BYTES;              // [stage][column block][key][128 B]
    int64_t *sums = reinterpret_cast<int64_t *>(smem_raw + (smem0 - smem_u32(smem_raw)));
    volatile int *abort_flag = &abort_word;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    auto full = [&](int s) { return bar(s); };
    auto empty = [&](int s) { return bar(C::STAGES + s); };
    auto q_ready = [&](int h) { return bar(2 * C::STAGES + h); };
    auto s_full = [&](int h) { return bar(2 * C::STAGES + 2 + h); };
    auto p_ready = [&](int h) { return bar(2 * C::STAGES + 4 + h); };
    auto o_full = [&](int h) { return bar(2 * C::STAGES + 6 + h); };
    const uint32_t drain_bar = bar(2 * C::STAGES + 8);

    if (threadIdx.x == 0) {
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(q_ready(h), 4);
            mbar_init(s_full(h), 1);
            mbar_init(p_ready(h), 4);
            mbar_init(o_full(h), 1);
        }
        mbar_init(drain_bar, 1);
        fence_barrier_init();
        abort_word = 0;
    }
    if (warp == 9)
        tmem_alloc(smem_u32(&tmem_slot), TMEM_COLS);
    pdl_wait();
    pdl_launch_dependents();
    const paged::Work &w = p.work;
    paged::group_units<BM, BN>(w, warp, THREADS / 32, sums);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = tmem_slot;
    int64_t per_head = 0;
    for (int g = 0; g < (w.seqs.seqs + 31) / 32; ++g)
        per_head += sums[g];
    const int64_t units = per_head * w.kv_heads;
    const int worker = blockIdx.x, workers = gridDim.x;
    const int64_t base = units / workers, extra = units % workers;
    const int64_t u0 = worker * base + min(static_cast<int64_t>(worker), extra);
    const int64_t count = base + (worker < extra ? 1 : 0);
    Cursor cur;
    if (count > 0)
        cur.seek(w, sums, per_head, u0);
    __syncthreads();                                           // sums is read; its memory is Q's

    // The whole warp waits; false after a timeout anywhere in the block.
    auto wait = [&](uint32_t b, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_try_wait(b, parity)) ||
               warp_wait_bounded(b, parity, abort_flag, p.wait_limit_ns);
    };
    // S_h at column h * 128 (P_h in its first 64 columns), O_h behind them.
    auto s_tmem = [&](int h) { return tmem + h * 128; };
    auto o_tmem = [&](int h) { return tmem + 256 + h * 128; };
    auto parts_tiles = [&](int64_t left) {
        const int64_t n = cur.t.end - cur.tile;
        return static_cast<int>(n < left ? n : left);
    };
    auto halves_of = [&]() { return cur.v.qlen * w.group - cur.m * BM > HALF ? 2 : 1; };

    paged::PartHeader head[2] = {};
    int64_t left = count;
    if (warp == 8) {
        // ================================================ keys and values
        const int page = 1 << w.seqs.page_shift;
        const int box = min(page, BN), subs = BN / box, boxes = subs * C::CH;
        int st = 0;
        uint32_t ph = 0, armed = 0;                            // armed: stages in flight, as bits
        bool ok = true;
        while (ok && left > 0) {
            const int nt = parts_tiles(left);
            for (int j = 0; ok && j < nt; ++j) {
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
                for (int kv = 0; kv < 2; ++kv) {
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
                }
            }
            left -= nt;
            if (ok && left > 0)
                cur.next_item(w);
        }
        // a block that gave up leaves no copy in flight: a stage's last phase
        // is the one before its next fill
        if (!ok && lane == 0)
            for (int s = 0; s < C::STAGES; ++s)
                if ((armed >> s) & 1u)
                    drain_wait(full(s), s < st ? ph : ph ^ 1u, p.wait_limit_ns);
    } else if (warp == 9) {
        // ======================================================= products
        constexpr uint32_t S_IDESC = idesc_bf16(HALF, BN, false);
        constexpr uint32_t O_IDESC = idesc_bf16(HALF, D, true);
        int st = 0;
        uint32_t ph = 0, q_ph[2] = {0, 0}, p_ph[2] = {0, 0};
        bool ok = true;
        auto next_stage = [&]() {
            if (++st == C::STAGES) {
                st = 0;
                ph ^= 1u;
            }
        };
        auto scores = [&](int h, int stage) {
            const uint64_t a = smem_desc_k128_sw128(q_smem + h * C::Q_BYTES);
            const uint64_t b = smem_desc_k128_sw128(ring + stage * C::TILE_BYTES);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                // 16 channels are 32 bytes of a 128-byte row, 64 a column block
                const uint64_t off = (k >> 2) * (HALF * 128 / 16) + (k & 3) * 2;
                umma_bf16_ss(s_tmem(h), a + off, b + off, S_IDESC, k > 0);
            }
            umma_commit(s_full(h));
        };
        while (ok && left > 0) {
            const int nt = parts_tiles(left), nh = halves_of();
            int k_stage = st;
            ok = wait(full(st), ph);
            next_stage();
            for (int h = 0; ok && h < nh; ++h) {
                ok = wait(q_ready(h), q_ph[h]);
                q_ph[h] ^= 1u;
                tc_fence_after_sync();
                if (ok && lane == 0)
                    scores(h, k_stage);
            }
            if (ok && lane == 0)
                umma_commit(empty(k_stage));
            for (int j = 0; ok && j < nt; ++j) {
                const int v_stage = st;
                ok = wait(full(st), ph);
                next_stage();
                if (!ok)
                    break;
                const int key0 = (cur.tile + j) * BN;
                const int skip = max(cur.t.klo - key0, 0), upto = min(cur.t.khi - key0, BN);
                if (skip > 0 || upto < BN) {
                    // slots that hold no key of the sequence may hold anything,
                    // and 0 * NaN is NaN: their values become zeros
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
                for (int h = 0; ok && h < nh; ++h) {
                    ok = wait(p_ready(h), p_ph[h]);
                    p_ph[h] ^= 1u;
                    if (!ok)
                        break;
                    tc_fence_after_sync();
                    if (lane == 0) {
                        const uint64_t b =
                            smem_desc_mn_sw128(ring + v_stage * C::TILE_BYTES, BN * 128);
#pragma unroll
                        for (int k = 0; k < BN / 16; ++k)      // 16 keys: two 1024-byte atoms
                            umma_bf16_ts(o_tmem(h), s_tmem(h) + k * 8, b + k * (2048 / 16), O_IDESC,
                                         j > 0 || k > 0);
                        if (h == nh - 1)
                            umma_commit(empty(v_stage));
                        if (j + 1 == nt)
                            umma_commit(o_full(h));
                    }
                    __syncwarp();
                    if (j + 1 < nt) {
                        if (h == 0) {
                            k_stage = st;
                            ok = wait(full(st), ph);
                            next_stage();
                            if (!ok)
                                break;
                        }
                        if (lane == 0) {
                            scores(h, k_stage);
                            if (h == nh - 1)
                                umma_commit(empty(k_stage));
                        }
                        __syncwarp();
                    }
                }
            }
            left -= nt;
            if (ok && left > 0)
                cur.next_item(w);
        }
        if (lane == 0) {                                       // nothing in flight at the end
            umma_commit(drain_bar);
            drain_wait(drain_bar, 0u, p.wait_limit_ns);
        }
    } else {
        // ======================================================== softmax
        const int h = warp >> 2;
        const int r = h * HALF + (warp & 3) * 32 + lane;       // row of the item
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_addr = s_tmem(h) + lane_off, o_addr = o_tmem(h) + lane_off;
        uint32_t s_ph = 0, o_ph = 0;
        bool ok = true;
        while (ok && left > 0) {
            const int nt = parts_tiles(left);
            const bool from_start = cur.tile == cur.t.begin;
            const bool to_end = cur.tile + nt == cur.t.end;
            const int rows = min(BM, cur.v.qlen * w.group - cur.m * BM);
            const int slot = 2 * worker + (from_start ? 1 : 0);
            const bool whole = from_start && to_end;
            if (!whole)
                head[from_start ? 1 : 0] = paged::PartHeader{to_end ? 2 : 1, cur.s, cur.m, cur.h};
            if (h < halves_of()) {
                const int rr = cur.m * BM + r;
                const int tok = rr / w.group;
                const int hq = cur.h * w.group + rr - tok * w.group;
                const int seen_hi = cur.v.kv - cur.v.qlen + tok;     // last key the row sees
                const int64_t row = cur.v.q0 + tok;
                {
                    const uint4 *src =
                        reinterpret_cast<const uint4 *>(p.q + row * p.q_stride + hq * D);
                    const uint32_t dst = q_smem + h * C::Q_BYTES + (r - h * HALF) * 128;
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 x = r < rows ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         dst + (c >> 3) * (HALF * 128) + (((c & 7) ^ (r & 7)) << 4)),
                                     "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w)
                                     : "memory");
                    }
                    fence_proxy_async();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(q_ready(h));
                }
                // keys that every row of this warp sees: tiles inside need no mask
                const int all_hi = __shfl_sync(0xffffffffu, seen_hi, 0);
                const int all_lo =
                    w.window > 0 ? __shfl_sync(0xffffffffu, seen_hi, 31) - w.window + 1 : 0;
                float m = -INFINITY, l = 0.0f;
                for (int j = 0; j < nt; ++j) {
                    if (!wait(s_full(h), s_ph)) {
                        ok = false;
                        break;
                    }
                    s_ph ^= 1u;
                    tc_fence_after_sync();
                    uint32_t s[BN];
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c)
                        tmem_ld_32x32b_x32(s_addr + c * 32,
                                           *reinterpret_cast<uint32_t(*)[32]>(s + c * 32));
                    tmem_ld_wait();
                    const int key0 = (cur.tile + j) * BN;
                    if (key0 + BN - 1 > all_hi || key0 < all_lo) {
                        const int hi = seen_hi - key0;
                        const int lo = w.window > 0 ? hi - w.window : -1;
#pragma unroll
                        for (int i = 0; i < BN; ++i)
                            if (i > hi || i <= lo)
                                s[i] = 0xff800000u;
                    }
                    float top = -INFINITY;
#pragma unroll
                    for (int i = 0; i < BN; i += 2)
                        top = fmaxf(top, fmaxf(__uint_as_float(s[i]), __uint_as_float(s[i + 1])));
                    top *= p.scale_log2;
                    const bool raise = top > m + RESCALE_AT;           // also from -inf
                    if (__any_sync(0xffffffffu, raise)) {
                        const float f = raise ? exp2_approx(m - top) : 1.0f;
                        if (raise)
                            m = top;
                        l *= f;
                        if (j > 0) {
#pragma unroll
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t o[32];
                                tmem_ld_32x32b_x32(o_addr + c * 32, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tmem_st_32x32b_x32(o_addr + c * 32, o);
                            }
                        }
                    }
                    const float sub = m == -INFINITY ? 0.0f : m;
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c) {
                        uint32_t e[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float a = exp2_approx(
                                fmaf(__uint_as_float(s[c * 32 + 2 * i]), p.scale_log2, -sub));
                            const float b = exp2_approx(
                                fmaf(__uint_as_float(s[c * 32 + 2 * i + 1]), p.scale_log2, -sub));
                            sum[i & 3] += a + b;
                            e[i] = pack_bf16(a, b);
                        }
                        tmem_st_x16(s_addr + c * 16, e);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tmem_st_wait();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(p_ready(h));
                }
                if (!ok || !wait(o_full(h), o_ph)) {
                    ok = false;
                    break;
                }
                o_ph ^= 1u;
                tc_fence_after_sync();
                const float f = whole ? inv_sum(l) : 1.0f;
                const int64_t at = static_cast<int64_t>(slot) * p.parts.row_cap + r;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(o_addr + c * 32, o);
                    tmem_ld_wait();
                    if (r < rows && whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(p.y + row * p.y_stride + hq * D +
                                                               c * 32);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t x[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                x[k] = pack_bf16(__uint_as_float(o[8 * i + 2 * k]) * f,
                                                 __uint_as_float(o[8 * i + 2 * k + 1]) * f);
                            dst[i] = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                    } else if (r < rows) {
                        uint4 *dst = reinterpret_cast<uint4 *>(p.parts.o + at * D + c * 32);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            dst[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
                if (r < rows) {
                    if (!whole)
                        p.parts.ml[at] = make_float2(m, l);
                    else if (p.lse != nullptr)
                        p.lse[row * p.q_heads + hq] = lse_of(m, l);
                }
            }
            left -= nt;
            if (left > 0)
                cur.next_item(w);
        }
        if (!ok)
            head[0].state = head[1].state = 0;                 // no part that could be merged
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 9) {
        tmem_relinquish();
        tmem_dealloc(tmem, TMEM_COLS);
    }
    if (threadIdx.x == 0) {
        if (abort_word)
            head[0].state = head[1].state = 0;
        p.parts.headers[2 * worker] = head[0];
        p.parts.headers[2 * worker + 1] = head[1];
    }
}

}  // namespace chunk
}  // namespace attn
}  // namespace bitlinear
