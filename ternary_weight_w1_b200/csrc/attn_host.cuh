// Host side of the operators on the paged key/value cache: argument checks,
// kernel choice and launches. Included by bitlinear.cu after its launch
// helpers; the C ABI functions are declared in include/bitlinear.h.
#pragma once

#include "row_set.cuh"

namespace {

constexpr int kAttnMaxGrid = 192;                    // SMs that a launch uses at most
constexpr int64_t kAttnMaxSeqs = 32 * paged::MAX_GROUPS;
constexpr int64_t kAttnMaxKeys = int64_t(1) << 30;   // page slots of a sequence
constexpr int64_t kAttnMaxRows = int64_t(1) << 30;   // tokens * query heads

// Rows of the queries or of the tensors beside them: a stride that keeps every
// row 16-byte aligned and apart from the next.
int check_rows(const void *p, int64_t stride, int64_t width)
{
    if (p == nullptr)
        return BITLINEAR_ERR_ARG;
    if (stride < width)
        return BITLINEAR_ERR_SHAPE;
    if (!aligned(p, 16) || stride % 8 != 0)
        return BITLINEAR_ERR_ALIGN;
    return BITLINEAR_OK;
}

// The shape checks of a cache and its sequences, without the pointers.
int check_paged_shape(int64_t tokens, int64_t seqs, int64_t q_heads, int64_t kv_heads,
                      int64_t head_dim)
{
    if (tokens < 0 || seqs < 0 || q_heads < 1 || kv_heads < 1)
        return BITLINEAR_ERR_ARG;
    if ((head_dim != 64 && head_dim != 128) || q_heads % kv_heads != 0 || q_heads > 65536 ||
        tokens > kAttnMaxRows / q_heads || seqs > kAttnMaxSeqs)
        return BITLINEAR_ERR_SHAPE;
    return BITLINEAR_OK;
}

int check_paged(int64_t tokens, int64_t q_heads, const bitlinear_kv_cache *c,
                const bitlinear_seqs *s, bool *empty)
{
    *empty = false;
    if (c == nullptr || s == nullptr || c->pages < 1 || s->table_cols < 1)
        return BITLINEAR_ERR_ARG;
    int rc = check_paged_shape(tokens, s->seqs, q_heads, c->kv_heads, c->head_dim);
    if (rc != BITLINEAR_OK)
        return rc;
    if (c->page < 16 || c->page > 256 || (c->page & (c->page - 1)) != 0 ||
        s->table_cols > kAttnMaxKeys / c->page ||
        c->pages > (INT_MAX - 512) / (c->kv_heads * c->page))
        return BITLINEAR_ERR_SHAPE;
    if (tokens == 0 || s->seqs == 0) {
        *empty = true;
        return BITLINEAR_OK;
    }
    if (c->k_dev == nullptr || c->v_dev == nullptr || s->q_start_dev == nullptr ||
        s->kv_len_dev == nullptr || s->page_table_dev == nullptr)
        return BITLINEAR_ERR_ARG;
    if (!aligned(c->k_dev, 16) || !aligned(c->v_dev, 16) || !aligned(s->q_start_dev, 4) ||
        !aligned(s->kv_len_dev, 4) || !aligned(s->page_table_dev, 4))
        return BITLINEAR_ERR_ALIGN;
    return BITLINEAR_OK;
}

int log2_of(int64_t v)
{
    int n = 0;
    while ((int64_t(1) << n) < v)
        ++n;
    return n;
}

paged::Divide divide_by(int64_t d)
{
    if (d == 1)
        return paged::Divide{0, -1};
    const int s = log2_of(d);
    return paged::Divide{static_cast<uint32_t>(((uint64_t(1) << (31 + s)) + d - 1) / d), s - 1};
}

paged::Seqs device_seqs(const bitlinear_kv_cache &c, const bitlinear_seqs &s, int64_t tokens)
{
    return paged::Seqs{s.q_start_dev,
                       s.kv_len_dev,
                       s.page_table_dev,
                       static_cast<int>(s.seqs),
                       static_cast<int>(s.table_cols),
                       static_cast<int>(tokens),
                       log2_of(c.page),
                       static_cast<int>(c.pages)};
}

// ------------------------------------------------------------ rope + append

template <int D>
cudaError_t launch_rope(const rope::Params &p, bool interleaved, int grid, cudaStream_t st)
{
    return launch(interleaved ? rope::rope_append_kernel<D, true>
                              : rope::rope_append_kernel<D, false>,
                  dim3(grid), dim3(rope::THREADS), 0, st, p);
}

// ---------------------------------------------------------------- attention

// A cache as a 2-D tensor {head_dim, pages * kv_heads * page} of bf16, boxed
// as {64 channels, box_rows} with the 128-byte swizzle: one box is a run of
// box_rows slots of one page and key head, 64 channels of each.
bool make_map_cache(CUtensorMap *map, const void *ptr, const bitlinear_kv_cache &c,
                    uint32_t box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr)
        return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.head_dim),
                                static_cast<cuuint64_t>(c.pages * c.kv_heads * c.page)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(c.head_dim) * 2};
    const cuuint32_t box[2] = {64, box_rows};
    const cuuint32_t estride[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides,
              box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries as a 3-D tensor {head_dim, q_heads, tokens}, boxed as {64
// channels, the heads of a group, `tokens` tokens}: the rows of half an item.
bool make_map_q(CUtensorMap *map, const attn::Params &p, int64_t head_dim, int tokens)
{
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr)
        return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim),
                                static_cast<cuuint64_t>(p.q_heads),
                                static_cast<cuuint64_t>(p.work.seqs.tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_dim) * 2,
                                   static_cast<cuuint64_t>(p.q_stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.work.group),
                               static_cast<cuuint32_t>(tokens)};
    const cuuint32_t estride[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(p.q), dims, strides,
              box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The parts of one attention kernel inside the workspace: headers, maxima and
// sums, accumulators, for two slots a worker.
size_t parts_layout(int64_t workers, int64_t row_cap, int64_t head_dim, bool flags, char *base,
                    paged::Parts *out)
{
    const size_t hb = round_up(static_cast<size_t>(2 * workers) * sizeof(paged::PartHeader), 256);
    const size_t mb = round_up(static_cast<size_t>(2 * workers * row_cap) * sizeof(float2), 256);
    const size_t ob = round_up(static_cast<size_t>(2 * workers * row_cap * head_dim) * 4, 256);
    const size_t fb =
        flags ? round_up(static_cast<size_t>(16 * workers) * sizeof(uint64_t), 256) : 0;
    if (out != nullptr) {
        out->headers = reinterpret_cast<paged::PartHeader *>(base);
        out->ml = reinterpret_cast<float2 *>(base + hb);
        out->o = reinterpret_cast<float *>(base + hb + mb);
        out->flags = flags ? reinterpret_cast<uint64_t *>(base + hb + mb + ob) : nullptr;
        out->row_cap = static_cast<int>(row_cap);
    }
    return hb + mb + ob + fb;
}

constexpr int kRowsKernelMax = 32;                   // rows of the rows kernel's largest item

// Rows up to which a sequence is better off in the rows kernel. 32 sequences of
// 4000 keys, rows kernel / chunk kernel: 32 rows on each of 10 key heads of 64
// channels 78 / 117 us, 20 rows on each of 5 of 128 channels 114 / 74 us, 32 rows
// 119 / 74 us, 16 rows 70 / 73 us. Two row tiles of 128 channels are more than a
// thread's registers hold, and half an item of the chunk kernel keeps up with HBM
// there. The rule looks at the rows alone, so it is not the best one for few
// sequences: four of 32 rows of 64 channels are 46 / 37.
constexpr int64_t rows_kernel_rows(int64_t head_dim) { return head_dim == 64 ? 32 : 16; }

// Workspace: the parts of the rows kernel, then those of the chunk kernel, which
// a call of no more rows than that never reaches.
struct AttnLayout {
    paged::Parts rows, chunk;
    size_t bytes;
};

AttnLayout attn_layout(int64_t rows, int64_t head_dim, char *base)
{
    AttnLayout l{};
    const int blocks = head_dim == 64 ? attn::rows::Cfg<64>::BLOCKS : attn::rows::Cfg<128>::BLOCKS;
    l.bytes = parts_layout(kAttnMaxGrid * blocks * attn::rows::WARPS,
                           std::min<int64_t>(rows, kRowsKernelMax), head_dim, false, base, &l.rows);
    if (rows > rows_kernel_rows(head_dim))
        l.bytes += parts_layout(kAttnMaxGrid, std::min<int64_t>(rows, 2 * attn::chunk::HALF),
                                head_dim, true, base + l.bytes, &l.chunk);
    return l;
}

template <int D>
int launch_merge(const attn::Params &p, int workers, bool chunk, const DeviceInfo &dev,
                 cudaStream_t st)
{
    const attn::MergeParams m{p.parts, p.y, p.y_stride, p.lse, p.q_heads, p.work, workers};
    // one wave of blocks, the items' rows dealt to them
    const int x = (workers + attn::MERGE_WARPS - 1) / attn::MERGE_WARPS;
    const int rows = std::min(p.work.item_rows, p.parts.row_cap);
    const dim3 grid(x, std::max(1, std::min(rows, 2 * dev.sms / x))), block(attn::MERGE_THREADS);
    return launch_status(launch(chunk ? attn::chunk::join_kernel<D> : attn::merge_kernel<D>, grid,
                                block, 0, st, m));
}

template <int D, int MT>
int run_attn_rows(attn::Params p, const bitlinear_kv_cache &cache, const DeviceInfo &dev,
                  cudaStream_t st)
{
    constexpr int smem = attn::rows::Cfg<D>::SMEM_BYTES;
    p.work.item_rows = 16 * MT;
    p.work.full = p.work.half = 1;
    p.work.start = 0;
    attn::Maps maps{};
    const uint32_t box = static_cast<uint32_t>(std::min<int64_t>(cache.page, attn::rows::BN));
    if (!make_map_cache(&maps.k, cache.k_dev, cache, box) ||
        !make_map_cache(&maps.v, cache.v_dev, cache, box))
        return BITLINEAR_ERR_CUDA;
    const int grid = std::min(dev.sms, kAttnMaxGrid) * attn::rows::Cfg<D>::BLOCKS;
    cudaError_t e = allow_smem<attn::rows::attn_rows_kernel<D, MT>>(dev.id, smem);
    if (e == cudaSuccess)
        e = launch(attn::rows::attn_rows_kernel<D, MT>, dim3(grid), dim3(attn::rows::THREADS),
                   static_cast<size_t>(smem), st, maps, p);
    const int rc = launch_status(e);
    return rc != BITLINEAR_OK ? rc : launch_merge<D>(p, grid * attn::rows::WARPS, false, dev, st);
}

// A number for every launch of the chunk kernel in this process: even, and
// counted from a place that no other memory content is likely to hold (the time
// of the first launch, spread over 64 bits by a multiplication).
uint64_t next_nonce()
{
    static std::atomic<uint64_t> next{
        static_cast<uint64_t>(std::chrono::system_clock::now().time_since_epoch().count()) *
            0x9E3779B97F4A7C15ull & ~uint64_t(1)};
    return next.fetch_add(2);
}

template <int D>
int run_attn_chunk(attn::Params p, const bitlinear_kv_cache &cache, const DeviceInfo &dev,
                   cudaStream_t st)
{
    constexpr int smem = attn::chunk::Cfg<D>::SMEM_BYTES;
    const int tokens = attn::chunk::HALF / p.work.group;       // of half an item
    p.work.item_rows = 2 * tokens * p.work.group;
    // A tile takes 2.2 us with both halves at work, 1.3 us with one (measured,
    // 128 channels); an item besides its tiles (its queries, its first scores, its
    // output) 2.5 us. A step of one 1021-token chunk and 47 single tokens takes
    // 91 us with an item's start at 0 units, 88 at 3, 86 at 5, 87 at 8; a
    // 2048-token prompt 48.5, 46.9, 47.9 and 48.0; windowed prompts 227, 218, 217
    // and 220.
    p.work.full = 5;
    p.work.half = 3;
    p.work.start = 5;
    attn::Maps maps{};
    CUtensorMap q_map;
    if (!make_map_q(&q_map, p, D, tokens))
        return BITLINEAR_ERR_CUDA;
    const uint32_t box = static_cast<uint32_t>(std::min<int64_t>(cache.page, attn::chunk::BN));
    if (!make_map_cache(&maps.k, cache.k_dev, cache, box) ||
        !make_map_cache(&maps.v, cache.v_dev, cache, box))
        return BITLINEAR_ERR_CUDA;
    const int grid = std::min(dev.sms, kAttnMaxGrid);
    // at most so many items, of so many tiles (the lengths are known on the device only)
    const double items = (static_cast<double>(p.work.seqs.tokens) / (2 * tokens) +
                          static_cast<double>(p.work.seqs.seqs)) * p.work.kv_heads;
    const double keys = static_cast<double>(p.work.seqs.table_cols) * cache.page;
    const double seen = p.work.window > 0 ? std::min(keys, p.work.window + 2.0 * tokens) : keys;
    const double units = items * ((seen / attn::chunk::BN + 2) * p.work.full + p.work.start);
    p.join_limit_ns = attn::chunk::join_wait_ns(p.wait_limit_ns, units / grid);
    cudaError_t e = allow_smem<attn::chunk::attn_chunk_kernel<D>>(dev.id, smem);
    if (e == cudaSuccess)
        e = launch(attn::chunk::attn_chunk_kernel<D>, dim3(grid), dim3(attn::chunk::THREADS),
                   static_cast<size_t>(smem), st, maps, q_map, p);
    const int rc = launch_status(e);
    return rc != BITLINEAR_OK ? rc : launch_merge<D>(p, grid, true, dev, st);
}

// The kernels of a step, by the rows (new tokens times query heads per key head)
// that its longest sequence can have. Few rows, and groups that no half item
// holds, take the rows kernel. Otherwise the chunk kernel takes all sequences in
// one launch, or, with 64 channels, only those of more rows than one item of the
// rows kernel, which takes the others: half an item of 64 channels reads the cache
// at half of HBM's rate. The second launch pays once there are three sequences
// and key heads per SM. One chunk and S single tokens behind 500 to 3000 keys, us
// in one launch / two:
//   64 channels, 10 heads  S = 31: 69 / 73    S = 63: 127 / 112  S = 127: 210 / 162
//   64 channels, 16 heads  S = 31: 98 / 84    S = 127: 320 / 210
//   128 channels, 5 heads  S = 31: 51 / 81    S = 63: 79 / 115   S = 127: 125 / 168
// With 64 tokens in the chunk; with 1024 (67 rows a sequence on average) and S = 63
// 186 / 153, with 1500 (191 rows) and S = 31 124 / 121.
template <int D>
int run_attention(attn::Params p, const bitlinear_kv_cache &cache, int64_t max_rows, char *ws,
                  const DeviceInfo &dev, cudaStream_t st)
{
    const int64_t rows = static_cast<int64_t>(p.work.seqs.tokens) * p.work.group;
    const AttnLayout layout = attn_layout(rows, D, ws);
    p.cache_rows = static_cast<int>(cache.pages * cache.kv_heads * cache.page);
    p.work.min_rows = 1;
    p.work.max_rows = INT_MAX;
    p.parts = layout.rows;
    if (max_rows <= 16)
        return run_attn_rows<D, 1>(p, cache, dev, st);
    if (max_rows <= rows_kernel_rows(D) || p.work.group > attn::chunk::HALF)
        return run_attn_rows<D, 2>(p, cache, dev, st);
    const int64_t seqs = p.work.seqs.seqs;
    if (D == 64 && p.work.group <= kRowsKernelMax && seqs * p.work.kv_heads >= 3 * dev.sms &&
        rows < 128 * seqs) {
        const bool small = p.work.group <= 16;
        p.work.max_rows = small ? 16 : 32;
        const int rc = small ? run_attn_rows<D, 1>(p, cache, dev, st)
                             : run_attn_rows<D, 2>(p, cache, dev, st);
        if (rc != BITLINEAR_OK)
            return rc;
        p.work.min_rows = p.work.max_rows + 1;
        p.work.max_rows = INT_MAX;
    }
    p.parts = layout.chunk;
    p.nonce = next_nonce();
    return run_attn_chunk<D>(p, cache, dev, st);
}

}  // namespace

extern "C" int bitlinear_rope_append(const void *q_dev, int64_t q_stride, const void *k_dev,
                                     int64_t k_stride, const void *v_dev, int64_t v_stride,
                                     int64_t tokens, int64_t q_heads,
                                     const bitlinear_kv_cache *cache, const bitlinear_seqs *seqs,
                                     const float *inv_freq_dev, int interleaved,
                                     const float *q_gain_dev, const float *k_gain_dev,
                                     float norm_eps, void *q_out_dev, int64_t q_out_stride,
                                     void *cuda_stream)
{
    bool empty = false;
    int rc = check_paged(tokens, q_heads, cache, seqs, &empty);
    if (rc != BITLINEAR_OK)
        return rc;
    const bool norm = q_gain_dev != nullptr || k_gain_dev != nullptr;
    if (norm && (!(norm_eps > 0.0f) || !(norm_eps <= FLT_MAX)))
        return BITLINEAR_ERR_ARG;
    if (interleaved != 0 && interleaved != 1)
        return BITLINEAR_ERR_ARG;
    if (empty)
        return BITLINEAR_OK;
    if (inv_freq_dev == nullptr)
        return BITLINEAR_ERR_ARG;
    const int64_t D = cache->head_dim;
    const struct { const void *p; int64_t stride, width; } rows[4] = {
        {q_dev, q_stride, q_heads * D},
        {k_dev, k_stride, cache->kv_heads * D},
        {v_dev, v_stride, cache->kv_heads * D},
        {q_out_dev, q_out_stride, q_heads * D}};
    for (const auto &r : rows) {
        rc = check_rows(r.p, r.stride, r.width);
        if (rc != BITLINEAR_OK)
            return rc;
    }
    if (!aligned(inv_freq_dev, 4) || !aligned(q_gain_dev, 4) || !aligned(k_gain_dev, 4))
        return BITLINEAR_ERR_ALIGN;
    // queries rotated where they stand are read and written by the same threads
    const RowSet out{q_out_dev, q_out_stride, q_heads * D};
    const bool in_place = q_out_dev == q_dev && (q_out_stride == q_stride || tokens == 1);
    if ((!in_place && share_memory(out, RowSet{q_dev, q_stride, q_heads * D}, tokens)) ||
        share_memory(out, RowSet{k_dev, k_stride, cache->kv_heads * D}, tokens) ||
        share_memory(out, RowSet{v_dev, v_stride, cache->kv_heads * D}, tokens))
        return BITLINEAR_ERR_ARG;
    DeviceInfo *dev = nullptr;
    rc = current_device(&dev);
    if (rc != BITLINEAR_OK)
        return rc;
    rope::Params p{};
    p.q = static_cast<const uint16_t *>(q_dev);
    p.k = static_cast<const uint16_t *>(k_dev);
    p.v = static_cast<const uint16_t *>(v_dev);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out = static_cast<uint16_t *>(q_out_dev);
    p.q_out_stride = q_out_stride;
    p.k_cache = static_cast<uint16_t *>(cache->k_dev);
    p.v_cache = static_cast<uint16_t *>(cache->v_dev);
    p.inv_freq = inv_freq_dev;
    p.q_gain = q_gain_dev;
    p.k_gain = k_gain_dev;
    p.eps = norm_eps;
    p.seqs = device_seqs(*cache, *seqs, tokens);
    p.q_heads = static_cast<int>(q_heads);
    p.kv_heads = static_cast<int>(cache->kv_heads);
    // a row per block until every SM has a few, then several
    p.per_block = static_cast<int>(
        std::min<int64_t>(rope::MAX_ROWS, std::max<int64_t>(1, tokens / (4 * dev->sms))));
    const int grid = static_cast<int>((tokens + p.per_block - 1) / p.per_block);
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    return launch_status(D == 64 ? launch_rope<64>(p, interleaved != 0, grid, st)
                                 : launch_rope<128>(p, interleaved != 0, grid, st));
}

extern "C" size_t bitlinear_workspace_bytes_attention(int64_t tokens, int64_t seqs,
                                                      int64_t q_heads, int64_t kv_heads,
                                                      int64_t head_dim)
{
    if (check_paged_shape(tokens, seqs, q_heads, kv_heads, head_dim) != BITLINEAR_OK)
        return SIZE_MAX;
    if (tokens == 0 || seqs == 0)
        return 0;
    return attn_layout(tokens * (q_heads / kv_heads), head_dim, nullptr).bytes;
}

namespace {

int paged_attention_impl(const void *q_dev, int64_t q_stride, int64_t tokens, int64_t q_heads,
                         const bitlinear_kv_cache *cache, const bitlinear_seqs *seqs, float scale,
                         int64_t window, int64_t max_q_len, void *y_dev, int64_t y_stride,
                         float *lse_dev_or_null, void *workspace_dev, size_t workspace_bytes,
                         void *cuda_stream, int stuck, uint64_t wait_limit_ns)
{
    bool empty = false;
    int rc = check_paged(tokens, q_heads, cache, seqs, &empty);
    if (rc != BITLINEAR_OK)
        return rc;
    if (!(scale > 0.0f) || !(scale <= FLT_MAX / 2) || window < 0 || max_q_len < 0)
        return BITLINEAR_ERR_ARG;
    if (empty)
        return BITLINEAR_OK;
    const int64_t D = cache->head_dim;
    rc = check_rows(q_dev, q_stride, q_heads * D);
    if (rc == BITLINEAR_OK)
        rc = check_rows(y_dev, y_stride, q_heads * D);
    if (rc != BITLINEAR_OK)
        return rc;
    if (!aligned(lse_dev_or_null, 4))
        return BITLINEAR_ERR_ALIGN;
    const size_t need = bitlinear_workspace_bytes_attention(tokens, seqs->seqs, q_heads,
                                                            cache->kv_heads, D);
    if (workspace_dev == nullptr || workspace_bytes < need)
        return BITLINEAR_ERR_WORKSPACE;
    if (!aligned(workspace_dev, 256))
        return BITLINEAR_ERR_ALIGN;
    if (share_memory(RowSet{y_dev, y_stride, q_heads * D}, RowSet{q_dev, q_stride, q_heads * D},
                     tokens))
        return BITLINEAR_ERR_ARG;
    DeviceInfo *dev = nullptr;
    rc = current_device(&dev);
    if (rc != BITLINEAR_OK)
        return rc;
    attn::Params p{};
    p.q = static_cast<const uint16_t *>(q_dev);
    p.y = static_cast<uint16_t *>(y_dev);
    p.q_stride = q_stride;
    p.y_stride = y_stride;
    p.lse = lse_dev_or_null;
    p.scale_log2 = scale * 1.44269504088896f;
    p.q_heads = static_cast<int>(q_heads);
    p.work.seqs = device_seqs(*cache, *seqs, tokens);
    p.work.kv_heads = static_cast<int>(cache->kv_heads);
    p.work.group = static_cast<int>(q_heads / cache->kv_heads);
    p.work.by_group = divide_by(p.work.group);
    p.work.window = static_cast<int>(std::min(window, kAttnMaxKeys));
    p.wait_limit_ns = wait_limit_ns;
    p.stuck = stuck;
    const int64_t longest = max_q_len > 0 ? std::min(max_q_len, tokens) : tokens;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    char *ws = static_cast<char *>(workspace_dev);
    return D == 64 ? run_attention<64>(p, *cache, longest * p.work.group, ws, *dev, st)
                   : run_attention<128>(p, *cache, longest * p.work.group, ws, *dev, st);
}

}  // namespace

extern "C" int bitlinear_paged_attention(const void *q_dev, int64_t q_stride, int64_t tokens,
                                         int64_t q_heads, const bitlinear_kv_cache *cache,
                                         const bitlinear_seqs *seqs, float scale, int64_t window,
                                         int64_t max_q_len, void *y_dev, int64_t y_stride,
                                         float *lse_dev_or_null, void *workspace_dev,
                                         size_t workspace_bytes, void *cuda_stream)
{
    return paged_attention_impl(q_dev, q_stride, tokens, q_heads, cache, seqs, scale, window,
                                max_q_len, y_dev, y_stride, lse_dev_or_null, workspace_dev,
                                workspace_bytes, cuda_stream, -1, kWaitLimitNs);
}

extern "C" int bitlinear_paged_attention_inject_timeout(
    const void *q_dev, int64_t q_stride, int64_t tokens, int64_t q_heads,
    const bitlinear_kv_cache *cache, const bitlinear_seqs *seqs, float scale, int64_t window,
    int64_t max_q_len, void *y_dev, int64_t y_stride, float *lse_dev_or_null, void *workspace_dev,
    size_t workspace_bytes, void *cuda_stream, int worker, int timeout_us)
{
    if (worker < 0 || timeout_us < 1 || timeout_us > 10 * 1000 * 1000)
        return BITLINEAR_ERR_ARG;
    return paged_attention_impl(q_dev, q_stride, tokens, q_heads, cache, seqs, scale, window,
                                max_q_len, y_dev, y_stride, lse_dev_or_null, workspace_dev,
                                workspace_bytes, cuda_stream, worker,
                                static_cast<uint64_t>(timeout_us) * 1000ull);
}

// ---------------------------------------------------------- attention block

namespace {

// Workspace of bitlinear_attn_forward: the projections' outputs and the
// attention's (behind q), then the scratch of one step at a time.
struct AttnBlock {
    size_t q, k, v, scratch, bytes;      // offsets, and the whole
    size_t scratch_bytes;
};

bool attn_block(int64_t M, int64_t K, int64_t seqs, int64_t q_heads, int64_t kv_heads,
                int64_t head_dim, AttnBlock *b)
{
    if (M < 0 || K < 1 || check_paged_shape(M, seqs, q_heads, kv_heads, head_dim) != BITLINEAR_OK)
        return false;
    const int64_t wide = q_heads * head_dim, narrow = kv_heads * head_dim;
    if (K % 128 != 0 || K > kMaxK || wide % 128 != 0 || wide > kMaxK)
        return false;
    bitlinear_problem pr[3] = {};
    for (int i = 0; i < 3; ++i)
        pr[i] = bitlinear_problem{nullptr, M, K, i == 0 ? wide : narrow, nullptr, 1.0f, nullptr};
    const size_t project = bitlinear_workspace_bytes_grouped(pr, 3);
    const size_t attend = bitlinear_workspace_bytes_attention(M, seqs, q_heads, kv_heads, head_dim);
    const size_t out = bitlinear_workspace_bytes(M, K, wide);
    if (project == SIZE_MAX || attend == SIZE_MAX || out == SIZE_MAX)
        return false;
    const size_t rows = static_cast<size_t>(M) * 2;
    b->q = 0;
    b->k = 2 * round_up(rows * wide, 256);
    b->v = b->k + round_up(rows * narrow, 256);
    b->scratch = b->v + round_up(rows * narrow, 256);
    b->scratch_bytes = std::max({project, attend, out});
    b->bytes = M == 0 ? 0 : b->scratch + b->scratch_bytes;
    return true;
}

}  // namespace

extern "C" size_t bitlinear_workspace_bytes_attn(int64_t M, int64_t K, int64_t seqs,
                                                 int64_t q_heads, int64_t kv_heads,
                                                 int64_t head_dim)
{
    AttnBlock b{};
    return attn_block(M, K, seqs, q_heads, kv_heads, head_dim, &b) ? b.bytes : SIZE_MAX;
}

extern "C" int bitlinear_attn_forward(const void *x_dev, bitlinear_dtype xdt, int64_t M, int64_t K,
                                      const bitlinear_projection *q, const bitlinear_projection *k,
                                      const bitlinear_projection *v, const bitlinear_projection *o,
                                      int64_t q_heads, const bitlinear_kv_cache *cache,
                                      const bitlinear_seqs *seqs, const float *inv_freq_dev,
                                      int interleaved, const float *q_head_gain_dev,
                                      const float *k_head_gain_dev, float norm_eps, float scale,
                                      int64_t window, int64_t max_q_len, void *y_dev,
                                      void *workspace_dev, size_t workspace_bytes,
                                      void *cuda_stream)
{
    if (q == nullptr || k == nullptr || v == nullptr || o == nullptr)
        return BITLINEAR_ERR_ARG;
    bool empty = false;
    int rc = check_paged(M, q_heads, cache, seqs, &empty);
    if (rc != BITLINEAR_OK)
        return rc;
    if (K < 1)
        return BITLINEAR_ERR_ARG;
    if (xdt != BITLINEAR_BF16 && xdt != BITLINEAR_FP32)
        return BITLINEAR_ERR_DTYPE;
    const int64_t D = cache->head_dim, wide = q_heads * D, narrow = cache->kv_heads * D;
    AttnBlock b{};
    if (!attn_block(M, K, seqs->seqs, q_heads, cache->kv_heads, D, &b))
        return BITLINEAR_ERR_SHAPE;
    const bool norm = q->gain_dev != nullptr;
    if ((k->gain_dev != nullptr) != norm || (v->gain_dev != nullptr) != norm)
        return BITLINEAR_ERR_ARG;
    if ((norm || o->gain_dev != nullptr || q_head_gain_dev != nullptr ||
         k_head_gain_dev != nullptr) &&
        (!(norm_eps > 0.0f) || !(norm_eps <= FLT_MAX)))
        return BITLINEAR_ERR_ARG;
    if (!(scale > 0.0f) || !(scale <= FLT_MAX / 2) || window < 0 || max_q_len < 0 ||
        (interleaved != 0 && interleaved != 1))
        return BITLINEAR_ERR_ARG;
    if (empty)
        return BITLINEAR_OK;
    const bitlinear_projection *const projections[4] = {q, k, v, o};
    for (const bitlinear_projection *p : projections) {
        if (p->packed_dev == nullptr)
            return BITLINEAR_ERR_ARG;
        if (!aligned(p->packed_dev, 16) || !aligned(p->gain_dev, 16))
            return BITLINEAR_ERR_ALIGN;
    }
    if (x_dev == nullptr || y_dev == nullptr || inv_freq_dev == nullptr)
        return BITLINEAR_ERR_ARG;
    if (!aligned(x_dev, 16) || !aligned(y_dev, 16) || !aligned(inv_freq_dev, 4) ||
        !aligned(q_head_gain_dev, 4) || !aligned(k_head_gain_dev, 4))
        return BITLINEAR_ERR_ALIGN;
    if (workspace_dev == nullptr || workspace_bytes < b.bytes)
        return BITLINEAR_ERR_WORKSPACE;
    if (!aligned(workspace_dev, 256))
        return BITLINEAR_ERR_ALIGN;

    char *ws = static_cast<char *>(workspace_dev);
    char *scratch = ws + b.scratch;
    void *qy = ws + b.q, *ky = ws + b.k, *vy = ws + b.v, *out = ws + b.k / 2;
    const bitlinear_problem pr[3] = {{x_dev, M, K, wide, q->packed_dev, q->gamma, qy},
                                     {x_dev, M, K, narrow, k->packed_dev, k->gamma, ky},
                                     {x_dev, M, K, narrow, v->packed_dev, v->gamma, vy}};
    const float *const gains[3] = {q->gain_dev, k->gain_dev, v->gain_dev};
    rc = norm ? bitlinear_forward_grouped_rmsnorm(pr, gains, 3, norm_eps, xdt, scratch,
                                                  b.scratch_bytes, cuda_stream)
              : bitlinear_forward_grouped_ws(pr, 3, xdt, scratch, b.scratch_bytes, cuda_stream);
    if (rc == BITLINEAR_OK)
        rc = bitlinear_rope_append(qy, wide, ky, narrow, vy, narrow, M, q_heads, cache, seqs,
                                   inv_freq_dev, interleaved, q_head_gain_dev, k_head_gain_dev,
                                   norm_eps, qy, wide, cuda_stream);
    if (rc == BITLINEAR_OK)
        rc = bitlinear_paged_attention(qy, wide, M, q_heads, cache, seqs, scale, window, max_q_len,
                                       out, wide, nullptr, scratch, b.scratch_bytes, cuda_stream);
    if (rc != BITLINEAR_OK)
        return rc;
    return forward_impl(out, BITLINEAR_BF16, M, wide, o->packed_dev, o->gamma, K, y_dev, scratch,
                        b.scratch_bytes, cuda_stream, nullptr, nullptr, nullptr,
                        BITLINEAR_PATH_AUTO, 0, o->gain_dev, norm_eps);
}
