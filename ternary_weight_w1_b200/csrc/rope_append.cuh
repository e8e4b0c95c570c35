// Rotation of the step's queries and keys by their positions, optionally
// RMS-normalised per head first, with the keys and values stored into the
// pages of their sequences.
//
// For a row at position p and the pair (a, b) of channels that share the
// frequency f: a' = a cos(p f) - b sin(p f), b' = b cos(p f) + a sin(p f).
// With gains, a head x becomes (x r) g first, r = 1 / sqrt(mean x^2 + eps).
//
// The kernel reads and writes every element once and is bound by memory for
// prompts and by its launch for a few tokens. A block takes `per_block` rows:
// its warps find the rows' sequences and compute the rows' cosines and sines
// once into shared memory (the head count is what shares them). A thread keeps
// 16 channels, 8 c .. and D / 2 + 8 c .., which are eight whole pairs in either
// order, and takes them of every head of its share, so a row's cosines and sines
// are read from shared memory once per thread, a pair never leaves a thread, and a
// head's sum of squares is a shuffle over D / 16 threads. Its next heads are on
// their way to shared memory meanwhile, each thread's to its own place, so no
// barrier is needed. The angle p f is taken in double and reduced by whole turns
// there: at position 10^5 an fp32 product would already be off by several
// thousandths of a turn. sinf and cosf then see |angle| <= pi.
//
// 17800 rows of 64 + 2 x 8 heads of 128 channels with norms, interleaved: 141 us,
// 5.2 TB/s of the 728 MB; 64% of the issue slots are taken, so memory and
// instructions bound it together. (The next heads in registers instead of shared
// memory 163 us; scalar instead of paired fp32 arithmetic and one stage 183 us.)
// One token 3.4 us, 61 tokens 4.3 us, most of it the call on the host.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "paged.cuh"

namespace bitlinear {
namespace rope {

constexpr int THREADS = 128;
constexpr int MAX_ROWS = 8;            // rows of a block
constexpr int STAGES = 6;              // units that a thread has in flight, and one

struct Params {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;   // elements from row to row
    uint16_t *q_out;
    int64_t q_out_stride;
    uint16_t *k_cache, *v_cache;
    const float *inv_freq;                  // [D / 2]
    const float *q_gain, *k_gain;           // [D] or null
    float eps;
    paged::Seqs seqs;
    int q_heads, kv_heads;
    int per_block;
};

// The sequence of row t: the one whose rows hold it, or -1. A warp narrows
// q_start[1 ..] by 32 probes at a time to the first entry above t.
__device__ __forceinline__ int find_seq(const paged::Seqs &q, int t)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = q.seqs;                 // the first entry above t is among [lo, lo + n]
    while (n > 0) {
        const int step = (n + 31) / 32;
        const int at = lo + min((lane + 1) * step, n) - 1;      // last entry of the lane's part
        const unsigned above = __ballot_sync(0xffffffffu, __ldg(q.q_start + 1 + at) > t);
        if (above == 0)
            return -1;                      // behind the last sequence
        const int part = __ffs(above) - 1;
        lo += part * step;
        n = min(step, n - part * step);
        if (step == 1)
            break;
    }
    return __ldg(q.q_start + lo) <= t ? lo : -1;
}

// eight bf16 as four pairs of fp32
__device__ __forceinline__ void unpack8(const uint4 &raw, uint64_t *v)
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

__device__ __forceinline__ uint4 pack8(const uint64_t *v)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        unpair(v[i], a, b);
        const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
        w[i] = *reinterpret_cast<const uint32_t *>(&x);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Shared arrays of eight pairs for each of T threads are kept in 16-byte pieces,
// piece q of thread c at (q * T + c) * 16, so that neighbours read neighbouring
// pieces. Element e of thread c:
template <int T>
__device__ __forceinline__ int piece_at(int c, int e)
{
    return ((e >> 2) * T + c) * 4 + (e & 3);
}

// pairs 2 q, 2 q + 1 of thread c
template <int T>
__device__ __forceinline__ void load_pairs(const float *p, int c, int q, uint64_t *v)
{
    const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(p + (q * T + c) * 4);
    v[0] = x.x;
    v[1] = x.y;
}

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS) rope_append_kernel(const Params p)
{
    constexpr int TPH = D / 16;             // threads per head
    constexpr int HALF = D / 2;
    constexpr int HPB = THREADS / TPH;      // heads a pass of the block
    // A row's factors as the products below take them, in pieces (piece_at):
    // cosines and sines of the thread's eight pairs, or for interleaved pairs
    // each cosine twice and each sine as (-sin, sin).
    __shared__ __align__(16) float cosines[MAX_ROWS][INTERLEAVED ? D : HALF];
    __shared__ __align__(16) float sines[MAX_ROWS][INTERLEAVED ? D : HALF];
    __shared__ __align__(16) float gains[2][D];         // of the queries, of the keys
    __shared__ uint4 staged[STAGES][2][THREADS];        // a thread's own next units
    __shared__ int64_t slot[MAX_ROWS];      // a row's first element in the caches, -1: none
    __shared__ int posn[MAX_ROWS];          // a row's position, -1: none

    pdl_wait();
    pdl_launch_dependents();
    const int t0 = blockIdx.x * p.per_block;
    const int rows = min(p.per_block, p.seqs.tokens - t0);
    for (int i = threadIdx.x; i < 2 * D; i += THREADS) {
        const float *gain = i < D ? p.q_gain : p.k_gain;
        if (gain != nullptr) {
            // channel e of a head belongs to thread c as its element j
            const int e = i % D;
            const int c = e % HALF / 8, j = e % 8 + e / HALF * 8;
            gains[i / D][piece_at<TPH>(c, j)] = __ldg(gain + e);
        }
    }
    for (int r = threadIdx.x >> 5; r < rows; r += THREADS / 32) {
        const int t = t0 + r;
        const int s = find_seq(p.seqs, t);
        if ((threadIdx.x & 31) == 0) {
            int pos = -1;
            int64_t at = -1;
            if (s >= 0) {
                // A row before position 0 has no place. Nor has any row of a sequence
                // with a value out of range: cut to what exists, it would put the
                // row in another token's.
                paged::View v;
                if (paged::read_view(p.seqs, s, v))
                    pos = max(v.kv - (v.q0 + v.qlen - t), -1);
                else
                    paged::fault_index();
            }
            if (pos >= 0) {
                const int page = paged::page_of(p.seqs, s, pos >> p.seqs.page_shift);
                const int size = 1 << p.seqs.page_shift;
                if (page >= 0)
                    at = (static_cast<int64_t>(page) * p.kv_heads * size + (pos & (size - 1))) * D;
            }
            posn[r] = pos;
            slot[r] = at;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * HALF; i += THREADS) {
        const int r = i / HALF, f = i % HALF;
        if (posn[r] < 0)
            continue;
        constexpr double TURN = 6.283185307179586476925;
        const double angle = posn[r] * static_cast<double>(__ldg(p.inv_freq + f));
        const float a = static_cast<float>(angle - rint(angle * (1.0 / TURN)) * TURN);
        const float co = cosf(a), si = sinf(a);
        if (INTERLEAVED) {
            // pair f is channels 2 f and 2 f + 1 of one 16-byte chunk
            const int c = f / 4 % TPH, j = f % 4 + f / 4 / TPH * 4;
            cosines[r][piece_at<TPH>(c, 2 * j)] = cosines[r][piece_at<TPH>(c, 2 * j + 1)] = co;
            sines[r][piece_at<TPH>(c, 2 * j)] = -si;
            sines[r][piece_at<TPH>(c, 2 * j + 1)] = si;
        } else {
            const int c = f / 8, j = f % 8;
            cosines[r][piece_at<TPH>(c, j)] = co;
            sines[r][piece_at<TPH>(c, j)] = si;
        }
    }
    __syncthreads();

    const int heads = p.q_heads + 2 * p.kv_heads;
    const int64_t head_step = static_cast<int64_t>(D) << p.seqs.page_shift;
    const int c = threadIdx.x % TPH;
    const int passes = (heads + HPB - 1) / HPB;
    const int units = rows * passes;        // head h0 + pass * HPB of a row, row after row
    const int h0 = threadIdx.x / TPH;
    // where unit (r, h) of this thread is read; null when there is none
    auto source = [&](int r, int h) -> const uint16_t * {
        if (h >= heads || posn[r] < 0)
            return nullptr;
        const int64_t t = t0 + r;
        return h < p.q_heads ? p.q + t * p.q_stride + h * D
               : h < p.q_heads + p.kv_heads
                   ? p.k + t * p.k_stride + (h - p.q_heads) * D
                   : p.v + t * p.v_stride + (h - p.q_heads - p.kv_heads) * D;
    };
    int fr = 0, fh = h0, fn = 0;            // next unit to fetch
    auto fetch = [&]() {
        if (fn < units) {
            const uint16_t *src = source(fr, fh);
            if (src != nullptr) {
                const uint32_t dst = smem_u32(&staged[fn % STAGES][0][threadIdx.x]);
                cp_async16(dst, src + 8 * c);
                cp_async16(dst + THREADS * 16, src + HALF + 8 * c);
            }
            ++fn;
            fh += HPB;
            if (fh >= passes * HPB) {
                fh = h0;
                ++fr;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i)
        fetch();
    constexpr int FACTORS = INTERLEAVED ? 8 : 4;        // pairs of cosines (sines)
    uint64_t co[FACTORS], si[FACTORS];
    for (int r = 0, n = 0; r < rows; ++r) {
        const int64_t t = t0 + r;
        const int64_t at = slot[r];
#pragma unroll
        for (int q = 0; q < FACTORS / 2; ++q) {
            load_pairs<TPH>(cosines[r], c, q, co + 2 * q);
            load_pairs<TPH>(sines[r], c, q, si + 2 * q);
        }
        for (int h = h0; h < passes * HPB; h += HPB, ++n) {
            fetch();
            asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
            // a head's threads share r and h, so they skip it together
            if (h >= heads || posn[r] < 0)
                continue;
            uint4 lo = staged[n % STAGES][0][threadIdx.x];
            uint4 hi = staged[n % STAGES][1][threadIdx.x];
            const bool is_q = h < p.q_heads, is_v = h >= p.q_heads + p.kv_heads;
            if (!is_v) {
                uint64_t x[8];
                unpack8(lo, x);
                unpack8(hi, x + 4);
                if ((is_q ? p.q_gain : p.k_gain) != nullptr) {
                    uint64_t ss2 = mul2(x[0], x[0]);
#pragma unroll
                    for (int j = 1; j < 8; ++j)
                        ss2 = fma2(x[j], x[j], ss2);
                    float ss, other;
                    unpair(ss2, ss, other);
                    ss += other;
                    const unsigned mask = (TPH == 8 ? 0xffu : 0xfu)
                                          << ((threadIdx.x & 31) & ~(TPH - 1));
#pragma unroll
                    for (int o = TPH / 2; o > 0; o >>= 1)
                        ss += __shfl_xor_sync(mask, ss, o);
                    const float rs = __fdiv_rn(1.0f, __fsqrt_rn(ss * (1.0f / D) + p.eps));
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint64_t g[2];
                        load_pairs<TPH>(gains[is_q ? 0 : 1], c, q, g);
                        x[2 * q] = mul2(mul2(x[2 * q], pair(rs, rs)), g[0]);
                        x[2 * q + 1] = mul2(mul2(x[2 * q + 1], pair(rs, rs)), g[1]);
                    }
                }
                if constexpr (INTERLEAVED) {
                    // (a, b) (cos, cos) + (b, a) (-sin, sin)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float a, b;
                        unpair(x[j], a, b);
                        x[j] = fma2(pair(b, a), si[j], mul2(x[j], co[j]));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint64_t minus = si[j] ^ 0x8000000080000000ull;
                        const uint64_t u = fma2(x[4 + j], minus, mul2(x[j], co[j]));
                        x[4 + j] = fma2(x[j], si[j], mul2(x[4 + j], co[j]));
                        x[j] = u;
                    }
                }
                lo = pack8(x);
                hi = pack8(x + 4);
            }
            if (is_q || at >= 0) {
                uint16_t *dst =
                    is_q ? p.q_out + t * p.q_out_stride + h * D
                         : is_v ? p.v_cache + at + (h - p.q_heads - p.kv_heads) * head_step
                                : p.k_cache + at + (h - p.q_heads) * head_step;
                *reinterpret_cast<uint4 *>(dst + 8 * c) = lo;
                *reinterpret_cast<uint4 *>(dst + HALF + 8 * c) = hi;
            }
        }
    }
}

}  // namespace rope
}  // namespace bitlinear
