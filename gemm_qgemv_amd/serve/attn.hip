// attn.hip -- entry point of attention over the paged 4-bit cache: checks,
// the choice of kernel and of the split of the tokens, launches.
#include "kv_host.hpp"

#include <cmath>

#include <algorithm>

#include "attn_few.hpp"
#include "attn_join.hpp"
#include "attn_rows.hpp"

namespace {

// A call's launch geometry: a pure function of sizes known on the host.
struct AttnPlan {
    int rows;              // query rows of a workgroup: 16 or 32 (attn_few_kernel), 64 or 128 (attn_rows_kernel)
    int64_t slots;         // tile slots
    int tile, step;        // tokens of a tile, and of a workgroup's round of tiles
    int nsplit;
    int32_t chunk;

    // at most `most` splits of `tokens` tokens, of whole rounds. A few rounds
    // stay in one split: the join would take longer (one row of 4 heads of 128
    // float32 channels: 2 rounds 10.9 us, 11.6 split, 3 rounds 13.8 and 12.3; 40
    // rows: 3 rounds 12.5 and 12.1, 4 rounds 15.0 and 11.9)
    void split(int64_t tokens, int64_t most)
    {
        const int64_t rounds = (tokens + step - 1) / step;
        most = std::max<int64_t>(most, 1);
        most = rounds <= (rows <= 32 ? 2 : 3) ? 1 : std::min(most, rounds);
        chunk = static_cast<int32_t>((rounds + most - 1) / most * step);
        nsplit = static_cast<int>((tokens + chunk - 1) / chunk);
    }
};

constexpr int few_or_rows_tile(int dim, int rows)
{
    return rows <= 32 ? qg::few_tile_tokens(dim) : qg::rows_tile_tokens(dim);
}

AttnPlan plan_attn(const qg_kv_cache &c, int batch, int64_t total_q, int64_t max_q, int64_t max_kv, int q_heads)
{
    const int group = q_heads / c.kv_heads;
    const int64_t most = std::min(max_q, total_q) * group;
    AttnPlan a;
    a.rows = most <= 16 ? 16 : most <= 32 ? 32 : most <= 64 || c.head_dim == 256 ? 64 : 128;
    a.slots = total_q * group / a.rows + batch;
    a.tile = few_or_rows_tile(c.head_dim, a.rows);
    a.step = a.tile * (a.rows == 16 ? 4 : a.rows == 32 ? 2 : 1);
    // two workgroups on every compute unit; four where decoding requests may
    // differ in length (64 requests of 1024 to 8192 tokens: 109 us at two, 90
    // at four, 88 at eight; one request of 131071: 44.6 at two, 45.4 at four)
    const int64_t tiles = std::max<int64_t>(1, total_q * group / a.rows);
    const int64_t have = std::max(tiles, std::min<int64_t>(batch, total_q)) * c.kv_heads;
    const int64_t aim = (a.rows == 16 && batch > 1 ? 4 : 2) * kComputeUnits;
    const int64_t want = std::max<int64_t>(1, (aim + have / 2) / have);
    // n splits take a workgroup rounds / n rounds, of 2 us or so, and n partial
    // results of every row written and read, at some terabytes a second: the
    // least sum is at a root (1280 rows of 128 float32 channels, 4000 tokens:
    // 31 us in 21 splits, 32 in 32; decoding stays far below)
    const double rounds = static_cast<double>(ceil_div(max_kv, a.step));
    const double best = std::sqrt(rounds * 2e6 / (static_cast<double>(total_q) * q_heads * c.head_dim));
    const int64_t most_splits = std::min<int64_t>({want, std::llround(best), qg::kMaxSplits});
    // few splits of requests that may differ in length, half a round longer each:
    // the last ones, which start last, are then short and even out the end (64
    // requests as above: 90 us, 93 with all alike; to 14000 tokens, 16 requests:
    // 41 and 47)
    const bool even_out = a.rows <= 32 && batch > 1 && most_splits > 1 && most_splits <= 8;
    a.split(max_kv + (even_out ? most_splits * a.step / 2 : 0), most_splits);
    return a;
}

// With a window a tile of rows sees at most window + rows tokens, from a first
// one that is rounded down to a tile: no more splits, of fewer tokens.
void narrow_plan(AttnPlan &a, int64_t max_kv, int64_t window)
{
    if (window < max_kv) a.split(std::min<int64_t>(max_kv, window + a.rows) + a.tile, a.nsplit);
}

size_t attn_workspace(const AttnPlan &a, const qg_kv_cache &c, int64_t total_q, int q_heads)
{
    if (a.nsplit == 1) return 0;
    return align256(static_cast<size_t>(total_q) * q_heads * a.nsplit * (c.head_dim + 2) * 4);
}

int check_attn_sizes(const qg_kv_cache &c, int batch, int64_t total_q, int64_t max_q, int64_t max_kv, int q_heads)
{
    if (batch < 1 || batch > 65535 || total_q < 1 || total_q > 0x7fffffffLL || max_q < 1 || max_kv < 1 ||
        max_kv > (int64_t(1) << 30) || q_heads < 1 || q_heads > 1024 || q_heads % c.kv_heads != 0)
        return QG_ERR_SHAPE;
    const AttnPlan a = plan_attn(c, batch, total_q, max_q, max_kv, q_heads);
    const int64_t rows = total_q * q_heads;
    return a.slots * c.kv_heads > kMaxWorkgroups || rows > 0x7fffffffLL ? QG_ERR_SHAPE : QG_OK;
}

template <auto KERNEL>
void launch_with_lds(size_t lds, dim3 grid, const qg::AttnParams &p, hipStream_t s)
{
    allow_lds<KERNEL>(lds);
    hipLaunchKernelGGL(KERNEL, grid, dim3(qg::kAttnThreads), lds, s, p);
}

template <typename T, int D, int R>
void launch_attn(const AttnPlan &a, const qg::AttnParams &p, hipStream_t s)
{
    const dim3 grid(static_cast<unsigned>(a.slots * p.kv.heads), static_cast<unsigned>(a.nsplit));
    if constexpr (R <= 32) launch_with_lds<qg::attn_few_kernel<T, D, R / 16>>(qg::few_lds_bytes<D>(), grid, p, s);
    else launch_with_lds<qg::attn_rows_kernel<T, D, R / 64>>(sizeof(qg::RowsLds<D>), grid, p, s);
    if (a.nsplit == 1) return;
    constexpr int TOK = few_or_rows_tile(D, R);
    const int64_t rows = p.total_q * p.q_heads;
    // a wave a row where splits are few (64 ragged requests: 89.5 us, 91.5 with a
    // workgroup a row; one row of 32 heads after 131071 tokens, 64 splits: 45.9, 44.8
    // with a workgroup)
    if (a.nsplit <= 16)
        hipLaunchKernelGGL((qg::attn_join_kernel<T, D, R, TOK, 1>), dim3(static_cast<unsigned>(ceil_div(rows, 4))), dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((qg::attn_join_kernel<T, D, R, TOK, 4>), dim3(static_cast<unsigned>(rows)), dim3(256), 0, s, p);
}

template <typename T, int D>
void launch_attn_dim(const AttnPlan &a, const qg::AttnParams &p, hipStream_t s)
{
    if (a.rows == 16) launch_attn<T, D, 16>(a, p, s);
    else if (a.rows == 32) launch_attn<T, D, 32>(a, p, s);
    else if (a.rows == 64) launch_attn<T, D, 64>(a, p, s);
    else if constexpr (D <= 128) launch_attn<T, D, 128>(a, p, s);
}

template <typename T>
void launch_attn_type(const AttnPlan &a, const qg::AttnParams &p, hipStream_t s)
{
    if (p.kv.dim == 64) launch_attn_dim<T, 64>(a, p, s);
    else if (p.kv.dim == 128) launch_attn_dim<T, 128>(a, p, s);
    else launch_attn_dim<T, 256>(a, p, s);
}

}  // namespace

extern "C" {

size_t qkv_attn_workspace_bytes(const qg_kv_cache *cache, int batch, int64_t total_q, int64_t max_q,
                                int64_t max_kv, int q_heads)
{
    if (!cache || check_geometry(*cache) != QG_OK) return 0;
    if (check_attn_sizes(*cache, batch, total_q, max_q, max_kv, q_heads) != QG_OK) return 0;
    return attn_workspace(plan_attn(*cache, batch, total_q, max_q, max_kv, q_heads), *cache, total_q, q_heads);
}

int qkv_attn(int dtype, const void *q, int64_t q_stride, const qg_kv_cache *cache,
             const int32_t *block_table, int64_t table_stride, const int32_t *cu_q,
             const int32_t *kv_len, int batch, int64_t total_q, int64_t max_q, int64_t max_kv,
             int q_heads, float scale, int64_t window, void *out, int64_t out_stride, float *lse,
             void *ws, size_t ws_bytes, hipStream_t stream)
{
    if (!known_dtype(dtype)) return QG_ERR_FORMAT;
    if (!q || !cache || !cache->data || !block_table || !cu_q || !kv_len || !out) return QG_ERR_NULL;
    int st = check_cache(*cache);
    if (st != QG_OK) return st;
    if ((st = check_attn_sizes(*cache, batch, total_q, max_q, max_kv, q_heads)) != QG_OK) return st;
    if (table_stride < 1 || table_stride > 0x7fffffffLL || max_kv > table_stride * cache->page_size || window < 0 ||
        !(scale > 0.0f) || !std::isfinite(scale * 1.5f))
        return QG_ERR_SHAPE;
    const int size = dtype == QG_F32 ? 4 : 2;
    const int64_t width = int64_t(q_heads) * cache->head_dim;
    for (const int64_t stride : {q_stride, out_stride})
        if (stride < width || stride > (int64_t(1) << 40) || stride * size % kAlign != 0) return QG_ERR_SHAPE;
    if (!aligned(q, kAlign) || !aligned(out, kAlign) || !aligned(block_table, 4) || !aligned(cu_q, 4) ||
        !aligned(kv_len, 4) || (lse && !aligned(lse, 4)))
        return QG_ERR_ALIGN;
    AttnPlan a = plan_attn(*cache, batch, total_q, max_q, max_kv, q_heads);
    if (window > 0) narrow_plan(a, max_kv, window);
    const size_t need = attn_workspace(a, *cache, total_q, q_heads);
    if (need > 0) {
        if (!ws || ws_bytes < need) return QG_ERR_WORKSPACE;
        if (!aligned(ws, kAlign)) return QG_ERR_ALIGN;
    }
    const Rows q_rows{reinterpret_cast<uintptr_t>(q), total_q, q_stride * size, width * size};
    const Rows out_rows{reinterpret_cast<uintptr_t>(out), total_q, out_stride * size, width * size};
    if (overlap(q_rows, out_rows)) return QG_ERR_ALIAS;
    const Range q_range = range_of(q, ((total_q - 1) * q_stride + width) * size);
    const Range inputs[4] = {range_of(cache->data, cache_bytes(*cache)), range_of(block_table, batch * table_stride * 4),
                             range_of(cu_q, (int64_t(batch) + 1) * 4), range_of(kv_len, int64_t(batch) * 4)};
    Range written[3];
    int nw = 0;
    written[nw++] = range_of(out, ((total_q - 1) * out_stride + width) * size);
    if (lse) written[nw++] = range_of(lse, total_q * q_heads * 4);
    if (need > 0) written[nw++] = range_of(ws, static_cast<int64_t>(need));
    if ((st = check_alias(inputs, 4, written, nw)) != QG_OK) return st;
    if ((st = check_alias(&q_range, 1, written + 1, nw - 1)) != QG_OK) return st;      // out: by rows, above

    (void)hipGetLastError();
    qg::AttnParams p{};
    p.q = q;
    p.q_stride = q_stride;
    p.kv = kv_view(*cache);
    p.table = block_table;
    p.table_stride = table_stride;
    p.cu_q = cu_q;
    p.kv_len = kv_len;
    p.batch = batch;
    p.total_q = total_q;
    p.max_kv = static_cast<int32_t>(max_kv);
    p.group = q_heads / cache->kv_heads;
    p.q_heads = q_heads;
    p.scale_log2e = scale * 1.44269504088896340736f;
    p.window = window > max_kv ? 0 : static_cast<int32_t>(window);
    p.out = out;
    p.out_stride = out_stride;
    p.lse = lse;
    p.nsplit = a.nsplit;
    p.chunk = a.chunk;
    if (a.nsplit > 1) {
        p.part_out = static_cast<float *>(ws);
        p.part_stat = p.part_out + total_q * q_heads * a.nsplit * cache->head_dim;
    }
    if (dtype == QG_F32) launch_attn_type<float>(a, p, stream);
    else launch_attn_type<uint16_t>(a, p, stream);
    return launch_status();
}

}  // extern "C"
