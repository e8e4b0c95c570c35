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
// once into shared memory (the head count is what shares them), then every
// thread takes 16 channels of one head, eight pairs, as two 16-byte loads, so
// a pair never leaves a thread and a head's sum of squares is a shuffle over
// D / 16 threads. The angle p f is taken in double and reduced by whole turns
// there: at position 10^5 an fp32 product would already be off by several
// thousandths of a turn. sinf and cosf then see |angle| <= pi.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "paged.cuh"

namespace bitlinear {
namespace rope {

constexpr int THREADS = 256;
constexpr int MAX_ROWS = 8;            // rows of a block

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

// eight bf16 at p as fp32
__device__ __forceinline__ void unpack8(const uint4 &raw, float *v)
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float *v)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS) rope_append_kernel(const Params p)
{
    constexpr int TPH = D / 16;             // threads per head
    constexpr int HALF = D / 2;
    __shared__ float cs[MAX_ROWS][2][HALF];
    __shared__ int64_t slot[MAX_ROWS];      // the row's element offset in the caches (head 0), -1: none
    __shared__ int posn[MAX_ROWS];          // the row's position, -1: no row of a sequence

    pdl_wait();
    pdl_launch_dependents();
    const int t0 = blockIdx.x * p.per_block;
    const int rows = min(p.per_block, p.seqs.tokens - t0);
    const int warp = threadIdx.x >> 5;
    if (warp < rows) {
        const int t = t0 + warp;
        const int s = find_seq(p.seqs, t);
        int pos = -1;
        int64_t at = -1;
        if (s >= 0 && (threadIdx.x & 31) == 0) {
            const paged::View v = paged::view(p.seqs, s);
            pos = v.kv - (v.q0 + v.qlen - t);
            if (pos >= 0) {
                const int page = paged::page_of(p.seqs, s, pos >> p.seqs.page_shift);
                const int size = 1 << p.seqs.page_shift;
                if (page >= 0)
                    at = (static_cast<int64_t>(page) * p.kv_heads * size + (pos & (size - 1))) * D;
            } else {
                pos = -1;                   // a row before position 0 has no place
            }
        }
        if ((threadIdx.x & 31) == 0) {
            posn[warp] = pos;
            slot[warp] = at;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * HALF; i += THREADS) {
        const int r = i / HALF, f = i % HALF;
        if (posn[r] < 0)
            continue;
        constexpr double TURN = 6.283185307179586476925;
        const double angle = static_cast<double>(posn[r]) * static_cast<double>(__ldg(p.inv_freq + f));
        const float a = static_cast<float>(angle - rint(angle / TURN) * TURN);
        cs[r][0][f] = cosf(a);
        cs[r][1][f] = sinf(a);
    }
    __syncthreads();

    const int heads = p.q_heads + 2 * p.kv_heads;
    const int64_t head_step = static_cast<int64_t>(D) << p.seqs.page_shift;
    for (int i = threadIdx.x; i < rows * heads * TPH; i += THREADS) {
        const int c = i % TPH;
        const int rh = i / TPH;
        const int r = rh / heads;
        const int h = rh - r * heads;
        // a head's threads share r and h, so they skip it together
        if (posn[r] < 0)
            continue;
        const int64_t t = t0 + r;
        const bool is_q = h < p.q_heads;
        const int hk = is_q ? 0 : (h - p.q_heads) % p.kv_heads;
        const bool is_v = h >= p.q_heads + p.kv_heads;
        const uint16_t *src = is_q ? p.q + t * p.q_stride + h * D
                                   : is_v ? p.v + t * p.v_stride + hk * D
                                          : p.k + t * p.k_stride + hk * D;
        uint16_t *dst;
        if (is_q)
            dst = p.q_out + t * p.q_out_stride + h * D;
        else
            dst = slot[r] < 0 ? nullptr : (is_v ? p.v_cache : p.k_cache) + slot[r] + hk * head_step;
        const int e0 = INTERLEAVED || is_v ? 16 * c : 8 * c;
        const int e1 = INTERLEAVED || is_v ? 16 * c + 8 : HALF + 8 * c;
        uint4 lo = *reinterpret_cast<const uint4 *>(src + e0);
        uint4 hi = *reinterpret_cast<const uint4 *>(src + e1);
        if (!is_v) {
            float x[16];
            unpack8(lo, x);
            unpack8(hi, x + 8);
            const float *gain = is_q ? p.q_gain : p.k_gain;
            if (gain != nullptr) {
                float ss = 0.0f;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    ss = fmaf(x[j], x[j], ss);
                const unsigned mask = (TPH == 8 ? 0xffu : 0xfu)
                                      << ((threadIdx.x & 31) & ~(TPH - 1));
#pragma unroll
                for (int o = TPH / 2; o > 0; o >>= 1)
                    ss += __shfl_xor_sync(mask, ss, o);
                const float rs = __fdiv_rn(
                    1.0f, __fsqrt_rn(ss * (1.0f / D) + p.eps));
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[j] = norm1(x[j], rs, __ldg(gain + e0 + j));
                    x[8 + j] = norm1(x[8 + j], rs, __ldg(gain + e1 + j));
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float &a = INTERLEAVED ? x[2 * j] : x[j];
                float &b = INTERLEAVED ? x[2 * j + 1] : x[8 + j];
                const float co = cs[r][0][8 * c + j], si = cs[r][1][8 * c + j];
                const float u = a * co - b * si;
                b = b * co + a * si;
                a = u;
            }
            lo = pack8(x);
            hi = pack8(x + 8);
        }
        if (dst != nullptr) {
            *reinterpret_cast<uint4 *>(dst + e0) = lo;
            *reinterpret_cast<uint4 *>(dst + e1) = hi;
        }
    }
}

}  // namespace rope
}  // namespace bitlinear
