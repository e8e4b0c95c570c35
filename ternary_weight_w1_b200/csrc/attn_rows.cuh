// Attention of few query rows over a paged cache (single tokens, drafted
// tokens): y_i = sum_j p_ij v_j, p_ij = softmax_j(scale q_i . k_j) over the
// keys j that row i sees.
//
// Every key and value is needed once per key head and each is used by a
// handful of rows (the query heads of the group times the new tokens), so the
// kernel is bound by the stream of the cache from HBM. Each warp works on its
// own: it owns a contiguous run of 32-key slices (paged.cuh), fetches them
// through its own ring of TMA stages, and computes with mma.sync m16n8k16,
// whose 16-row tile is the smallest that the tensor pipe offers; the rows of
// a group fill it, and a warp needs no barrier with any other warp. Tensor
// maps box the pages with the 128-byte swizzle, so ldmatrix reads keys and
// (transposed) values without bank conflicts.
//
// The softmax runs once over the keys: a row keeps its maximum m, its sum l
// and its accumulator o in fp32, all relative to m. m is raised only when a
// score passes it by more than 8 in log2 units: p <= 2^8 stays far inside
// fp32 and bf16, and the accumulators are rescaled a few times per row instead
// of once per slice. p is rounded to bf16 for the second product (relative
// 2^-8 at most, of random sign from key to key, so a row's error stays below
// the rounding of the output); the sum l takes p before that rounding.
//
// 96 sequences behind 500 to 9500 keys, 64 heads on 8 of 128 channels: 2.07 GB in
// 326 to 335 us, 6.2 to 6.4 TB/s, the rate of a plain copy; 61 sequences behind 1 to
// 4095 keys, 20 heads on 5: 362 MB in 72 us, of which 5 are the start and 5 the
// merge; one token behind 700: 10 us, the two launches. 24 sequences of five tokens,
// 40 heads on 10 of 64 channels: 49 us with two blocks an SM, 65 with one.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"
#include "paged.cuh"

namespace bitlinear {
namespace attn {

constexpr float RESCALE_AT = 8.0f;     // log2 units

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int c0, int c1,
                                            uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void fence_proxy_async()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

struct Params {
    const uint16_t *q;         // row t, head h at q + t * q_stride + h * D
    uint16_t *y;
    int64_t q_stride, y_stride;
    float *lse;                // [tokens][q_heads] or null
    float scale_log2;          // scale * log2(e)
    int q_heads;
    int cache_rows;            // pages * kv_heads * page: the first row behind the cache
    paged::Work work;
    paged::Parts parts;
    uint64_t wait_limit_ns;
    uint64_t join_limit_ns;    // of the chunk kernel's waits for other blocks
    int stuck;                 // worker whose first stage never fills (a test), or -1
    uint64_t nonce;            // even, another for every launch
};

struct Maps {
    CUtensorMap k, v;          // {D, cache_rows}, boxes {64, min(page, tile)}, 128-byte swizzle
};

// Finishes an item's row from its sum and accumulator scale: 1 / l, or 0 for
// a row that sees no key.
__device__ __forceinline__ float inv_sum(float l) { return l > 0.0f ? __fdividef(1.0f, l) : 0.0f; }

__device__ __forceinline__ float lse_of(float m, float l)
{
    return l > 0.0f ? (m + log2f(l)) * 0.693147180559945f : -INFINITY;
}

namespace rows {

constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int BN = 32;                 // keys of a slice

// One block an SM, or two for 64 channels: a slice then has half the bytes for
// nearly the same latency, and eight warps keep as many bytes in flight.
template <int D>
struct Cfg {
    static constexpr int BLOCKS = D == 64 ? 2 : 1;               // per SM
    static constexpr int RING_BYTES = 48 * 1024 / BLOCKS;        // of one warp
    static constexpr int HALVES = D / 64;
    static constexpr int HALF_BYTES = BN * 128;
    static constexpr int TENSOR_BYTES = HALVES * HALF_BYTES;     // the slice's keys (or values)
    static constexpr int STAGE_BYTES = 2 * TENSOR_BYTES;
    static constexpr int STAGES = RING_BYTES / STAGE_BYTES;
    static constexpr int SMEM_BYTES = 1024 + WARPS * RING_BYTES;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// MT 16-row tiles per item.
template <int D, int MT>
__global__ void __launch_bounds__(THREADS, Cfg<D>::BLOCKS)
    attn_rows_kernel(const __grid_constant__ Maps maps, const Params p)
{
    using C = Cfg<D>;
    constexpr int BM = 16 * MT;
    constexpr int KS = D / 16;             // k-steps of the score product
    constexpr int NT = D / 8;              // 8-channel tiles of the output
    using Cursor = paged::Cursor<BN>;

    extern __shared__ char smem_raw[];
    __shared__ int64_t sums[paged::MAX_GROUPS];
    __shared__ __align__(8) uint64_t bars[WARPS][C::STAGES];
    __shared__ int abort_word;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int worker = warp * gridDim.x + blockIdx.x;
    const int workers = WARPS * gridDim.x;
    volatile int *abort_flag = &abort_word;
    const uint32_t ring = ((smem_u32(smem_raw) + 1023u) & ~1023u) + warp * C::RING_BYTES;
    if (threadIdx.x == 0) {
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
        abort_word = 0;
    }
    if (lane == 0) {
        for (int i = 0; i < C::STAGES; ++i)
            mbar_init(smem_u32(&bars[warp][i]), 1 + (i == 0 && worker == p.stuck));
        fence_barrier_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    const paged::Work &w = p.work;
    Cursor cur;
    const int64_t count = paged::deal<BN>(w, worker, workers, sums, cur);

    paged::PartHeader head[2] = {};
    if (count > 0) {
        const int page = 1 << w.seqs.page_shift;
        const int box = min(page, BN);                 // rows of one TMA box
        const int subs = BN / box;                     // boxes of a slice and half
        Cursor ld = cur;

        // Lane i loads the slice's box i: tensor (k, v), half of the channels,
        // part of the rows. A box without a needed key, or of a page that the table
        // does not hold, starts behind the cache and is filled with zeros. The
        // pages of 32 slices are looked up at a time, one slice's a lane.
        const int boxes = 2 * C::HALVES * subs;
        int64_t loaded = 0, done = 0;
        int ld_stage = 0, stage = 0;
        uint32_t parity = 0;
        int first = 0, ahead = 0;                      // the slices looked up
        int ids[2] = {-1, -1};                         // (two pages a slice when they are of 16)
        auto load = [&]() {
            if (ld.tile - first >= ahead) {
                first = ld.tile;
                ahead = min(32, ld.t.end - first);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int key = (first + lane) * BN + i * box;
                    ids[i] = -1;
                    if (i < subs && key < ld.t.khi && key + box > ld.t.klo)
                        ids[i] = paged::page_of(w.seqs, ld.s, key >> w.seqs.page_shift);
                }
            }
            const int id0 = __shfl_sync(0xffffffffu, ids[0], ld.tile - first);
            const int id1 = __shfl_sync(0xffffffffu, ids[1], ld.tile - first);
            const int st = ld_stage;
            ld_stage = ld_stage + 1 == C::STAGES ? 0 : ld_stage + 1;
            const uint32_t bar = smem_u32(&bars[warp][st]);
            if (lane == 0)
                mbar_arrive_expect_tx(bar, C::STAGE_BYTES);
            __syncwarp();
            if (lane < boxes) {
                const int sub = lane % subs;
                const int half = (lane / subs) % C::HALVES;
                const bool is_v = lane >= subs * C::HALVES;
                const int key = ld.tile * BN + sub * box;
                const int id = sub == 0 ? id0 : id1;
                const int row = id < 0 ? p.cache_rows
                                       : ((id * w.kv_heads + ld.h) << w.seqs.page_shift) +
                                             (key & (page - 1));
                const uint32_t dst = ring + st * C::STAGE_BYTES + (is_v ? C::TENSOR_BYTES : 0) +
                                     half * C::HALF_BYTES + sub * box * 128;
                tma_load_2d(dst, is_v ? &maps.v : &maps.k, half * 64, row, bar);
            }
            if (++loaded < count && ++ld.tile == ld.t.end) {
                ld.next_item(w);
                ahead = 0;
                first = ld.tile;
            }
        };
        for (int i = 0; i < C::STAGES && loaded < count; ++i)
            load();

        bool ok = true;
        while (ok && done < count) {
            // ---- one item, or the part of it in this worker's run
            const bool from_start = cur.tile == cur.t.begin;
            const int rows = min(BM, cur.v.qlen * w.group - cur.m * BM);
            const int pos0 = cur.v.kv - cur.v.qlen;
            const int r_lo = lane >> 2;                // rows r_lo and r_lo + 8 of each 16-row tile
            uint32_t qf[MT][KS][4];
            int seen_hi[2 * MT];                       // last key the row sees
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = mt * 16 + e * 8 + r_lo;
                    const int rr = cur.m * BM + r;
                    const int tok = w.by_group(rr);
                    seen_hi[2 * mt + e] = pos0 + tok;
                    const uint32_t *src = reinterpret_cast<const uint32_t *>(
                        p.q + (cur.v.q0 + tok) * p.q_stride +
                        (cur.h * w.group + rr - tok * w.group) * D + (lane & 3) * 2);
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        qf[mt][ks][e] = r < rows ? __ldg(src + ks * 8) : 0u;
                        qf[mt][ks][2 + e] = r < rows ? __ldg(src + ks * 8 + 4) : 0u;
                    }
                }
            }
            float o[MT][NT][4];
            float m[2 * MT], l[2 * MT];
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
                m[i] = -INFINITY;
                l[i] = 0.0f;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[mt][n][i] = 0.0f;

            // keys every row of the item sees: slices inside need no mask
            const int all_hi = pos0 + w.by_group(cur.m * BM);
            const int all_lo = w.window > 0 ? cur.t.khi - w.window : 0;
            for (; done < count; ) {
                const uint32_t bar = smem_u32(&bars[warp][stage]);
                if (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity)) &&
                    !warp_wait_bounded(bar, parity, abort_flag, p.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                const uint32_t ks_base = ring + stage * C::STAGE_BYTES;
                const uint32_t vs_base = ks_base + C::TENSOR_BYTES;
                const int key0 = cur.tile * BN;
                if (key0 < cur.t.klo || key0 + BN > cur.t.khi) {
                    // slots that hold no key of the sequence may hold anything,
                    // and 0 * NaN is NaN: their values become zeros
                    const int key = key0 + lane;
                    if (key < cur.t.klo || key >= cur.t.khi) {
#pragma unroll
                        for (int i = 0; i < C::HALVES * 8; ++i)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             vs_base + (i >> 3) * C::HALF_BYTES + lane * 128 +
                                             (i & 7) * 16),
                                         "r"(0)
                                         : "memory");
                    }
                    fence_proxy_async();
                    __syncwarp();
                }

                // ---- scores of 16 MT rows and 32 keys
                float s[MT][4][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            s[mt][n][i] = 0.0f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
                    for (int np = 0; np < 2; ++np) {   // two 8-key tiles at a time
                        const int row = np * 16 + (lane & 7) + ((lane & 16) >> 1);
                        const int chunk = (ks & 3) * 2 + ((lane >> 3) & 1);
                        uint32_t b[4];
                        ldsm4(b, ks_base + (ks >> 2) * C::HALF_BYTES + row * 128 +
                                     ((chunk ^ (row & 7)) << 4));
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            mma_bf16(s[mt][2 * np], qf[mt][ks], b[0], b[1]);
                            mma_bf16(s[mt][2 * np + 1], qf[mt][ks], b[2], b[3]);
                        }
                    }
                }
                if (key0 + BN - 1 > all_hi || key0 < all_lo) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int n = 0; n < 4; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int key = key0 + n * 8 + (lane & 3) * 2 + (i & 1);
                                const int hi = seen_hi[2 * mt + (i >> 1)];
                                if (key > hi || (w.window > 0 && key <= hi - w.window))
                                    s[mt][n][i] = -INFINITY;
                            }
                }

                // ---- running maximum and sum
                float sub[2 * MT];
#pragma unroll
                for (int i = 0; i < 2 * MT; ++i) {
                    float top = -INFINITY;
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        top = fmaxf(top, fmaxf(s[i >> 1][n][2 * (i & 1)],
                                               s[i >> 1][n][2 * (i & 1) + 1]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    top *= p.scale_log2;
                    const bool raise = top > m[i] + RESCALE_AT;     // also from -inf
                    if (__any_sync(0xffffffffu, raise)) {
                        if (raise) {
                            const float f = exp2_approx(m[i] - top);
                            m[i] = top;
                            l[i] *= f;
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                o[i >> 1][n][2 * (i & 1)] *= f;
                                o[i >> 1][n][2 * (i & 1) + 1] *= f;
                            }
                        }
                    }
                    sub[i] = m[i] == -INFINITY ? 0.0f : m[i];
                }
                uint32_t pf[MT][2][4];                 // p as the second product's A operand
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        float e[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            e[i] = exp2_approx(
                                fmaf(s[mt][n][i], p.scale_log2, -sub[2 * mt + (i >> 1)]));
                        l[2 * mt] += e[0] + e[1];
                        l[2 * mt + 1] += e[2] + e[3];
                        pf[mt][n >> 1][(n & 1) * 2] = pack_bf16(e[0], e[1]);
                        pf[mt][n >> 1][(n & 1) * 2 + 1] = pack_bf16(e[2], e[3]);
                    }

                // ---- o += p v
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {       // 16 keys at a time
                    const int row = kk * 16 + (lane & 15);
#pragma unroll
                    for (int np = 0; np < NT / 2; ++np) {
                        const int chunk = (np & 3) * 2 + (lane >> 4);
                        uint32_t b[4];
                        ldsm4_t(b, vs_base + (np >> 2) * C::HALF_BYTES + row * 128 +
                                       ((chunk ^ (row & 7)) << 4));
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            mma_bf16(o[mt][2 * np], pf[mt][kk], b[0], b[1]);
                            mma_bf16(o[mt][2 * np + 1], pf[mt][kk], b[2], b[3]);
                        }
                    }
                }
                __syncwarp();                          // every lane has read the stage
                ++done;
                if (++stage == C::STAGES) {
                    stage = 0;
                    parity ^= 1u;
                }
                if (loaded < count)
                    load();
                if (++cur.tile == cur.t.end)
                    break;
            }
            if (!ok)
                break;

            // ---- the item's rows, or their part
            const bool to_end = cur.tile == cur.t.end;
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            }
            const int slot = 2 * worker + (from_start ? 1 : 0);
            const bool whole = from_start && to_end;
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
                const int r = (i >> 1) * 16 + (i & 1) * 8 + r_lo;
                if (r >= rows)
                    continue;
                if (whole) {
                    const int rr = cur.m * BM + r;
                    const int tok = w.by_group(rr);
                    const int hq = cur.h * w.group + rr - tok * w.group;
                    const float f = inv_sum(l[i]);
                    uint32_t *dst = reinterpret_cast<uint32_t *>(
                        p.y + (cur.v.q0 + tok) * p.y_stride + hq * D + (lane & 3) * 2);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        dst[n * 4] = pack_bf16(o[i >> 1][n][2 * (i & 1)] * f,
                                               o[i >> 1][n][2 * (i & 1) + 1] * f);
                    if (p.lse != nullptr && (lane & 3) == 0)
                        p.lse[static_cast<int64_t>(cur.v.q0 + tok) * p.q_heads + hq] =
                            lse_of(m[i], l[i]);
                } else {
                    const int64_t at = static_cast<int64_t>(slot) * p.parts.row_cap + r;
                    float2 *dst = reinterpret_cast<float2 *>(p.parts.o + at * D) + (lane & 3);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        dst[n * 4] = make_float2(o[i >> 1][n][2 * (i & 1)],
                                                 o[i >> 1][n][2 * (i & 1) + 1]);
                    if ((lane & 3) == 0)
                        p.parts.ml[at] = make_float2(m[i], l[i]);
                }
            }
            if (!whole)
                head[from_start ? 1 : 0] =
                    paged::PartHeader{rows, to_end ? 0 : 1, cur.v.q0, cur.h + w.kv_heads * cur.m};
            if (done < count)
                cur.next_item(w);
        }
        if (!ok) {
            // leave no copy in flight behind, and no part that could be merged
            for (; lane == 0 && done < loaded; ++done) {
                drain_wait(smem_u32(&bars[warp][stage]), parity, p.wait_limit_ns);
                if (++stage == C::STAGES) {
                    stage = 0;
                    parity ^= 1u;
                }
            }
            head[0].rows = head[1].rows = 0;
        }
    }
    if (lane < 2)
        p.parts.headers[2 * worker + lane] = lane == 0 ? head[0] : head[1];
}

}  // namespace rows

// ------------------------------------------------------------------- merge
//
// Joins the parts of the items that were split between workers: o = sum_i
// 2^(m_i - M) o_i and l likewise, M the largest m_i. A split item begins in some
// worker's second slot and goes on in the first slots of the workers behind it.
// Block (x, y) lists the split items of workers 8 x .. 8 x + 7, one a warp, and
// takes every gridDim.y-th of their row groups. A warp's lanes take D / 32
// channels each of a row and have eight parts in flight: of one row, or of two
// or four rows when the item has few parts. With many parts (a single token
// behind a long context) the parts of a row are spread over the block's warps,
// which are then added in a fixed order, so that repeated calls give the same
// bits.

constexpr int MERGE_WARPS = 8;
constexpr int MERGE_THREADS = MERGE_WARPS * 32;
struct MergeParams {
    paged::Parts parts;
    uint16_t *y;
    int64_t y_stride;
    float *lse;
    int q_heads;
    paged::Work work;
    int workers;
};

template <int D>
struct Merge {
    static constexpr int VEC = D / 32;                 // channels of a lane
    using Vec = typename std::conditional<VEC == 4, float4, float2>::type;

    const MergeParams &p;
    paged::PartHeader hd;
    int first, parts, lane, m;

    // part 0 is slot `first`, part i > 0 slot first + 2 i - 1
    __device__ __forceinline__ int64_t at(int i, int r) const
    {
        return static_cast<int64_t>(first + (i > 0 ? 2 * i - 1 : 0)) * p.parts.row_cap + r;
    }

    __device__ __forceinline__ Vec load(int i, int r) const
    {
        return *reinterpret_cast<const Vec *>(p.parts.o + at(i, r) * D + VEC * lane);
    }

    static __device__ __forceinline__ void add(float (&acc)[VEC], const Vec &x, float f)
    {
        const float *e = reinterpret_cast<const float *>(&x);
#pragma unroll
        for (int c = 0; c < VEC; ++c)
            acc[c] = fmaf(e[c], f, acc[c]);
    }

    __device__ __forceinline__ void store(int r, const float (&acc)[VEC], float top, float l) const
    {
        const int rr = m * p.work.item_rows + r;
        const int tok = p.work.by_group(rr);
        const int hq = (hd.hm - m * p.work.kv_heads) * p.work.group + rr - tok * p.work.group;
        const int64_t row = hd.row + tok;
        const float f = inv_sum(l);
        uint32_t *dst = reinterpret_cast<uint32_t *>(p.y + row * p.y_stride + hq * D + VEC * lane);
#pragma unroll
        for (int c = 0; c < VEC / 2; ++c)
            dst[c] = pack_bf16(acc[2 * c] * f, acc[2 * c + 1] * f);
        if (p.lse != nullptr && lane == 0)
            p.lse[row * p.q_heads + hq] = lse_of(top, l);
    }

    // Rows r .. r + 8 / NP of an item of at most NP parts: lane 8 i + j holds
    // part j of row i.
    template <int NP>
    __device__ __forceinline__ void few(int r) const
    {
        constexpr int ROWS = 8 / NP;
        const int i = lane >> 3, j = lane & 7;
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (i < ROWS && j < parts && r + i < hd.rows)
            ml = p.parts.ml[at(j, r + i)];
        Vec x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k % NP < parts && r + k / NP < hd.rows)
                x[k] = load(k % NP, r + k / NP);
        float top = ml.x;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float f = exp2_approx(ml.x - (top == -INFINITY ? 0.0f : top));
        float l = ml.y * f;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1)
            l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            float acc[VEC] = {};
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const float g = __shfl_sync(0xffffffffu, f, 8 * q + k);
                if (k < parts && r + q < hd.rows)
                    add(acc, x[q * NP + k], g);
            }
            const float t = __shfl_sync(0xffffffffu, top, 8 * q);
            const float s = __shfl_sync(0xffffffffu, l, 8 * q);
            if (r + q < hd.rows)
                store(r + q, acc, t, s);
        }
    }
};

// Lists the split items that begin in workers 8 x .. 8 x + 7, one a warp: their
// headers and numbers of parts (0: none begins there). Ends with a barrier.
__device__ __forceinline__ void list_items(const MergeParams &p, paged::PartHeader *begun,
                                           int *count)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wk = blockIdx.x * MERGE_WARPS + warp;
    paged::PartHeader hd{};
    if (wk < p.workers)
        hd = p.parts.headers[2 * wk + 1];
    int n = 1;
    // the following workers' first slots, 32 at a time, up to the last part
    for (int at = wk + 1;; at += 32) {
        paged::PartHeader next{};
        if (at + lane < p.workers)
            next = p.parts.headers[2 * (at + lane)];
        if (hd.rows == 0 || !hd.more) {
            n = 0;
            break;
        }
        const unsigned ends = __ballot_sync(0xffffffffu, next.rows == 0 || !next.more);
        if (ends == 0) {
            n += 32;
            continue;
        }
        const int last = __ffs(ends) - 1;
        // (an item whose last part is missing, as a worker gave up, is left out)
        n = __shfl_sync(0xffffffffu, next.rows, last) == 0 ? 0 : n + last + 1;
        break;
    }
    if (n > 0) {
        // a workspace that another call writes at the same time (which is not
        // allowed) may hold anything: no address comes from it unchecked
        const int64_t last =
            static_cast<int64_t>(hd.hm / p.work.kv_heads) * p.work.item_rows + hd.rows - 1;
        if (hd.rows < 0 || hd.rows > p.parts.row_cap || hd.hm < 0 || hd.row < 0 ||
            last >= (int64_t(1) << 31) ||
            hd.row + static_cast<int64_t>(p.work.by_group(static_cast<int>(last))) >=
                p.work.seqs.tokens) {
            paged::fault_index();
            n = 0;
        }
    }
    if (lane == 0) {
        begun[warp] = hd;
        count[warp] = n;
    }
    __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(MERGE_THREADS, 2) merge_kernel(const MergeParams p)
{
    using M = Merge<D>;
    __shared__ float partial[MERGE_WARPS][D];
    __shared__ paged::PartHeader begun[MERGE_WARPS];
    __shared__ int count[MERGE_WARPS];
    pdl_wait();
    pdl_launch_dependents();
    list_items(p, begun, count);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the items of few parts: groups of their rows, dealt to all warps
    for (int j = blockIdx.y * MERGE_WARPS + warp;; j += gridDim.y * MERGE_WARPS) {
        int i = 0, g = j, parts = 0;
        for (; i < MERGE_WARPS; ++i) {
            parts = count[i];
            const int group = parts <= 2 ? 4 : parts <= 4 ? 2 : 1;
            const int groups = parts == 0 || parts > 8 ? 0 : (begun[i].rows + group - 1) / group;
            if (g < groups)
                break;
            g -= groups;
        }
        if (i == MERGE_WARPS)
            break;
        M mg{p, begun[i], 2 * (static_cast<int>(blockIdx.x) * MERGE_WARPS + i) + 1, parts, lane, 0};
        mg.m = mg.hd.hm / p.work.kv_heads;
        if (parts <= 2)
            mg.template few<2>(g * 4);
        else if (parts <= 4)
            mg.template few<4>(g * 2);
        else
            mg.template few<8>(g);
    }
    // the others: a row's parts spread over the block
    for (int i = 0; i < MERGE_WARPS; ++i) {
        const int parts = count[i];
        if (parts <= 8)
            continue;
        M mg{p, begun[i], 2 * (static_cast<int>(blockIdx.x) * MERGE_WARPS + i) + 1, parts, lane, 0};
        mg.m = mg.hd.hm / p.work.kv_heads;
        const int rows = mg.hd.rows;
        // warps a row: as many as leave each about four parts
        const int spread = parts >= 32 ? 8 : parts >= 16 ? 4 : 2;
        const int sub = warp & (spread - 1);
        const int pass = MERGE_WARPS / spread;         // rows of the block at a time
        for (int r0 = blockIdx.y * pass; r0 < rows; r0 += gridDim.y * pass) {
            const int r = r0 + warp / spread;
            const bool live = r < rows;
            float2 ml = make_float2(-INFINITY, 0.0f);
            float top = -INFINITY;
            for (int i = lane; live && i < parts; i += 32) {
                ml = p.parts.ml[mg.at(i, r)];
                top = fmaxf(top, ml.x);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float base = top == -INFINITY ? 0.0f : top;
            float l = 0.0f;
            float acc[M::VEC] = {};
            for (int i0 = 0; i0 < parts; i0 += 32) {
                float f = 0.0f;
                if (live && i0 + lane < parts) {
                    if (parts > 32)
                        ml = p.parts.ml[mg.at(i0 + lane, r)];
                    f = exp2_approx(ml.x - base);
                    l = fmaf(ml.y, f, l);
                }
                const int n = min(32, parts - i0);
                for (int b = sub; b < n; b += 8 * spread) {
                    typename M::Vec x[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (live && b + k * spread < n)
                            x[k] = mg.load(i0 + b + k * spread, r);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float g = __shfl_sync(0xffffffffu, f, (b + k * spread) & 31);
                        if (live && b + k * spread < n)
                            M::add(acc, x[k], g);
                    }
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                l += __shfl_xor_sync(0xffffffffu, l, o);
            __syncthreads();                               // the sums before have been read
#pragma unroll
            for (int c = 0; c < M::VEC; ++c)
                partial[warp][M::VEC * lane + c] = acc[c];
            __syncthreads();
            if (live && sub == 0) {
                for (int k = 1; k < spread; ++k)
#pragma unroll
                    for (int c = 0; c < M::VEC; ++c)
                        acc[c] += partial[warp + k][M::VEC * lane + c];
                mg.store(r, acc, top, l);
            }
        }
    }
}

}  // namespace attn
}  // namespace bitlinear
