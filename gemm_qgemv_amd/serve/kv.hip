// kv.hip -- entry points of the paged 4-bit key/value cache: its size, the
// page plan of a step, append and read-back. Host-side checks and launches;
// the arithmetic is in plan.hpp and append.hpp.
#include "kv_host.hpp"

#include <algorithm>

#include "append.hpp"
#include "plan.hpp"

namespace {

// Rows of activations: `n` rows `stride` elements apart, `width` used.
int check_rows(int dtype, const void *p, int64_t stride, int64_t width)
{
    const int size = dtype == QG_F32 ? 4 : 2;
    if (stride < width || stride > (int64_t(1) << 40) || stride * size % kAlign != 0) return QG_ERR_SHAPE;
    return aligned(p, kAlign) ? QG_OK : QG_ERR_ALIGN;
}

Rows rows_of(int dtype, const void *p, int64_t stride, int64_t width, int64_t n)
{
    const int64_t size = dtype == QG_F32 ? 4 : 2;
    return Rows{reinterpret_cast<uintptr_t>(p), n, stride * size, width * size};
}

Range rows_range(int dtype, const void *p, int64_t stride, int64_t width, int64_t n)
{
    return range_of(p, ((n - 1) * stride + width) * (dtype == QG_F32 ? 4 : 2));
}

qg::AppendMap append_map(const qg_kv_cache &c)
{
    qg::AppendMap m;
    m.per_row = c.kv_heads * c.head_dim / 8;
    m.rows = std::max(1, qg::kAppendThreads / m.per_row);
    m.inv = 1.0f / static_cast<float>(m.per_row);
    return m;
}

// Launches over all rows, in pieces that a grid holds. `parts`: K and V in
// workgroups of their own (2) or together (1); side(p, i): K's and V's rows.
template <typename P, typename Side>
void launch_rows(void (*kernel)(P), P p, unsigned parts, int64_t element, Side side, hipStream_t stream)
{
    const int64_t n = p.n, most = kMaxWorkgroups * p.map.rows;
    for (int64_t first = 0; first < n; first += most) {
        p.n = std::min(n - first, most);
        const dim3 grid(static_cast<unsigned>(ceil_div(p.n, p.map.rows)), parts,
                        static_cast<unsigned>(ceil_div(p.map.per_row, qg::kAppendThreads)));
        hipLaunchKernelGGL(kernel, grid, dim3(qg::kAppendThreads), 0, stream, p);
        p.slots += p.n;
        for (int i = 0; i < 2; ++i)
            if (side(p, i)) side(p, i) += p.n * p.stride[i] * element;
    }
}

}  // namespace

extern "C" {

size_t qkv_cache_bytes(const qg_kv_cache *cache)
{
    if (!cache || check_geometry(*cache) != QG_OK) return 0;
    return static_cast<size_t>(cache_bytes(*cache));
}

int qkv_plan(const int32_t *len_old, const int32_t *keep, const int32_t *n_new, int batch,
             int page_size, int32_t *block_table, int64_t table_stride, int32_t *ring,
             int64_t ring_size, const int64_t *state_in, int64_t *state_out, int32_t *kv_len,
             int32_t *cu_q, int32_t *slots, int32_t *pos, int64_t total, int32_t *denied,
             hipStream_t stream)
{
    if (!len_old || !keep || !n_new || !block_table || !ring || !state_in || !state_out || !kv_len ||
        !cu_q || !denied || (total > 0 && (!slots || !pos)))
        return QG_ERR_NULL;
    if (batch < 1 || batch > QG_MAX_PLAN_BATCH || page_size < 1 || page_size > (1 << 20) ||
        (page_size & (page_size - 1)) != 0 || table_stride < 1 || table_stride > 0x7fffffffLL ||
        ring_size < 1 || ring_size > 0x7fffffffLL || total < 0 || total > 0x7fffffffLL)
        return QG_ERR_SHAPE;
    for (const void *p : {static_cast<const void *>(len_old), static_cast<const void *>(keep),
                          static_cast<const void *>(n_new), static_cast<const void *>(block_table),
                          static_cast<const void *>(ring), static_cast<const void *>(kv_len),
                          static_cast<const void *>(cu_q), static_cast<const void *>(slots),
                          static_cast<const void *>(pos), static_cast<const void *>(denied)})
        if (!aligned(p, 4)) return QG_ERR_ALIGN;
    if (!aligned(state_in, 8) || !aligned(state_out, 8)) return QG_ERR_ALIGN;
    const Range inputs[4] = {range_of(len_old, int64_t(batch) * 4), range_of(keep, int64_t(batch) * 4),
                             range_of(n_new, int64_t(batch) * 4), range_of(state_in, 16)};
    const Range written[8] = {range_of(block_table, batch * table_stride * 4), range_of(ring, ring_size * 4),
                              range_of(state_out, 16), range_of(kv_len, int64_t(batch) * 4),
                              range_of(cu_q, (int64_t(batch) + 1) * 4), range_of(denied, 4),
                              range_of(slots, total * 4), range_of(pos, total * 4)};
    const int st = check_alias(inputs, 4, written, 8);
    if (st != QG_OK) return st;

    (void)hipGetLastError();
    qg::PlanParams p{len_old, keep, n_new, batch, __builtin_ctz(static_cast<unsigned>(page_size)), block_table,
                     table_stride, ring, ring_size, state_in, state_out, kv_len, cu_q, slots, pos, total, denied};
    // two tokens a thread (each takes a chain of LDS reads to find its request;
    // every workgroup repeats the running sums; 65536 tokens of 512 requests: 13.3
    // us at eight, 6.7 at two); and a workgroup for eight requests, whose pages
    // may all come back though they get few tokens (64 requests, four of them
    // ended with some 1000 pages: 7.5 us with one workgroup, 4.2 with eight)
    const int64_t parts = std::max(ceil_div(total, qg::kPlanThreads * 2), ceil_div(batch, 8));
    const auto grid = static_cast<unsigned>(std::clamp<int64_t>(parts, 1, 256));
    const size_t lds = (3 * static_cast<size_t>(batch) + 1) * 4;
    allow_lds<qg::kv_plan_kernel>((3 * QG_MAX_PLAN_BATCH + 1) * 4);
    hipLaunchKernelGGL(qg::kv_plan_kernel, dim3(grid, 3), dim3(qg::kPlanThreads), lds, stream, p);
    return launch_status();
}

int qkv_append(int dtype, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
               const int32_t *slots, int64_t n, const qg_kv_cache *cache, hipStream_t stream)
{
    if (!known_dtype(dtype)) return QG_ERR_FORMAT;
    if (!cache || !cache->data) return QG_ERR_NULL;
    if (n > 0 && (!k || !v || !slots)) return QG_ERR_NULL;
    int st = check_cache(*cache);
    if (st != QG_OK) return st;
    if (n < 0 || n > 0x7fffffffLL) return QG_ERR_SHAPE;
    if (n == 0) return QG_OK;
    const int64_t width = int64_t(cache->kv_heads) * cache->head_dim;
    if ((st = check_rows(dtype, k, k_stride, width)) != QG_OK) return st;
    if ((st = check_rows(dtype, v, v_stride, width)) != QG_OK) return st;
    if (!aligned(slots, 4)) return QG_ERR_ALIGN;
    const Range inputs[3] = {rows_range(dtype, k, k_stride, width, n), rows_range(dtype, v, v_stride, width, n),
                             range_of(slots, n * 4)};
    const Range written[1] = {range_of(cache->data, cache_bytes(*cache))};
    if ((st = check_alias(inputs, 3, written, 1)) != QG_OK) return st;

    (void)hipGetLastError();
    qg::AppendParams p{{static_cast<const char *>(k), static_cast<const char *>(v)}, {k_stride, v_stride}, slots, n,
                       append_map(*cache), kv_view(*cache)};
    auto src = [](qg::AppendParams &q, int i) -> const char *& { return q.src[i]; };
    if (dtype == QG_F32) launch_rows(qg::kv_append_kernel<float>, p, 1, 4, src, stream);
    else launch_rows(qg::kv_append_kernel<uint16_t>, p, 1, 2, src, stream);
    return launch_status();
}

int qkv_read(int dtype, const qg_kv_cache *cache, const int32_t *slots, int64_t n, void *k,
             int64_t k_stride, void *v, int64_t v_stride, hipStream_t stream)
{
    if (!known_dtype(dtype)) return QG_ERR_FORMAT;
    if (!cache || !cache->data) return QG_ERR_NULL;
    if (n > 0 && (!slots || (!k && !v))) return QG_ERR_NULL;
    int st = check_cache(*cache);
    if (st != QG_OK) return st;
    if (n < 0 || n > 0x7fffffffLL) return QG_ERR_SHAPE;
    if (n == 0) return QG_OK;
    const int64_t width = int64_t(cache->kv_heads) * cache->head_dim;
    if (k && (st = check_rows(dtype, k, k_stride, width)) != QG_OK) return st;
    if (v && (st = check_rows(dtype, v, v_stride, width)) != QG_OK) return st;
    if (!aligned(slots, 4)) return QG_ERR_ALIGN;
    const Range inputs[2] = {range_of(cache->data, cache_bytes(*cache)), range_of(slots, n * 4)};
    for (const Range &w : {rows_range(dtype, k ? k : v, k ? k_stride : v_stride, width, n),
                           rows_range(dtype, v ? v : k, v ? v_stride : k_stride, width, n)})
        if ((st = check_alias(inputs, 2, &w, 1)) != QG_OK) return st;
    if (k && v && overlap(rows_of(dtype, k, k_stride, width, n), rows_of(dtype, v, v_stride, width, n))) return QG_ERR_ALIAS;

    (void)hipGetLastError();
    qg::ReadParams p{{static_cast<char *>(k), static_cast<char *>(v)}, {k_stride, v_stride}, slots, n, append_map(*cache), kv_view(*cache)};
    auto dst = [](qg::ReadParams &q, int i) -> char *& { return q.dst[i]; };
    if (dtype == QG_F32) launch_rows(qg::kv_read_kernel<float>, p, 2, 4, dst, stream);
    else launch_rows(qg::kv_read_kernel<uint16_t>, p, 2, 2, dst, stream);
    return launch_status();
}

}  // extern "C"
