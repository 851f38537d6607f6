// moe.hip -- entry points around the experts' products: router, sort by
// expert, way back.
#include "mx_host.hpp"

#include <algorithm>

#include "combine.hpp"
#include "route.hpp"

namespace {

// Logits of a lane up to which router and sort are one launch (the waves of a workgroup of
// 1024 threads have 128 registers).
constexpr int kFusedLogits = 16;

struct Sort {
    int64_t run;
    int runs;
};

// Runs of 2048 pairs, and no more of them than kSortMaxRuns.
Sort plan_sort(int64_t pairs)
{
    const int64_t unit = 64 * qg::kSortWaves;
    const int64_t run = std::max<int64_t>(qg::kSortSteps * unit, round_up(ceil_div(pairs, qg::kSortMaxRuns), unit));
    return Sort{run, static_cast<int>(std::max<int64_t>(1, ceil_div(pairs, run)))};
}

size_t sort_bytes(const Sort &s, int experts) { return s.runs == 1 ? 0 : align256(static_cast<size_t>(s.runs) * experts * 4); }

qg::SortParams sort_params(const Sort &s, const int32_t *ids, int64_t pairs, int experts, int32_t *offsets, int32_t *order, int32_t *slots,
                           void *ws)
{
    qg::SortParams p{};
    p.ids = ids;
    p.pairs = pairs;
    p.run = s.run;
    p.runs = s.runs;
    p.experts = experts;
    while ((experts >> p.bits) != 0) ++p.bits;       // numbers 0..experts
    p.counts = static_cast<int32_t *>(ws);
    p.offsets = offsets;
    p.order = order;
    p.slots = slots;
    return p;
}

size_t sort_lds(int experts) { return static_cast<size_t>(qg::sort_place_ints(experts)) * 4; }

void launch_sort(const qg::SortParams &p, hipStream_t stream)
{
    if (p.runs > 1)
        hipLaunchKernelGGL(qg::sort_count_kernel, dim3(static_cast<unsigned>(p.runs)), dim3(qg::kSortThreads), (static_cast<size_t>(p.experts) + 1) * 4,
                           stream, p);
    static std::atomic<uint64_t> asked{0};
    allow_dynamic_lds(reinterpret_cast<const void *>(&qg::sort_place_kernel), sort_lds(QMOE_MAX_EXPERTS), asked);
    hipLaunchKernelGGL(qg::sort_place_kernel, dim3(static_cast<unsigned>(p.runs)), dim3(qg::kSortThreads), sort_lds(p.experts), stream, p);
}

// Checks that the router and the plan share; `need` is the workspace's size.
int check_plan(const int32_t *ids, int64_t rows, int experts, int top, const int32_t *offsets, const int32_t *order, const int32_t *slots,
               const void *ws, size_t ws_bytes, size_t &need)
{
    if (!ids || !offsets || !order || !slots) return QG_ERR_NULL;
    if (!moe_sizes_ok(rows, experts, top)) return QG_ERR_SHAPE;
    for (const void *q : {static_cast<const void *>(ids), static_cast<const void *>(offsets), static_cast<const void *>(order),
                          static_cast<const void *>(slots)})
        if (!aligned(q, 4)) return QG_ERR_ALIGN;
    need = sort_bytes(plan_sort(rows * top), experts);
    if (need > 0) {
        if (!ws || ws_bytes < need) return QG_ERR_WORKSPACE;
        if (!aligned(ws, kAlign)) return QG_ERR_ALIGN;
    }
    return QG_OK;
}

template <typename T, int V>
void launch_route(const qg::RouteParams &p, const qg::SortParams &s, hipStream_t stream)
{
    // One workgroup for both, where the rows are no more than it takes at once.
    if constexpr (V <= kFusedLogits) {
        if (p.rows <= qg::kRouteSortRows && s.runs == 1) {
            static std::atomic<uint64_t> asked{0};
            allow_dynamic_lds(reinterpret_cast<const void *>(&qg::route_sort_kernel<T, V>), sort_lds(16 * V), asked);
            hipLaunchKernelGGL((qg::route_sort_kernel<T, V>), dim3(1), dim3(qg::kSortThreads), sort_lds(p.experts), stream, p, s);
            return;
        }
    }
    if (p.rows > 0)
        hipLaunchKernelGGL((qg::route_kernel<T, V>), dim3(static_cast<unsigned>(ceil_div(p.rows, qg::kRouteRows))), dim3(qg::kRouteThreads), 0, stream, p);
    launch_sort(s, stream);
}

template <typename T>
void launch_route(const qg::RouteParams &p, const qg::SortParams &s, hipStream_t stream)
{
    if (p.experts <= 64) launch_route<T, 4>(p, s, stream);
    else if (p.experts <= 128) launch_route<T, 8>(p, s, stream);
    else if (p.experts <= 256) launch_route<T, 16>(p, s, stream);
    else if (p.experts <= 512) launch_route<T, 32>(p, s, stream);
    else launch_route<T, 64>(p, s, stream);
}

}  // namespace

extern "C" {

size_t qmoe_plan_workspace_bytes(int64_t rows, int experts, int top)
{
    return moe_sizes_ok(rows, experts, top) ? sort_bytes(plan_sort(rows * top), experts) : 0;
}

int qmoe_plan(const int32_t *ids, int64_t rows, int experts, int top, int32_t *offsets, int32_t *order, int32_t *slots, void *ws,
              size_t ws_bytes, hipStream_t stream)
{
    size_t need = 0;
    int st = check_plan(ids, rows, experts, top, offsets, order, slots, ws, ws_bytes, need);
    if (st != QG_OK) return st;
    const int64_t pairs = rows * top;
    const Range in = range_of(ids, pairs * 4);
    const Range out[4] = {range_of(offsets, (int64_t(experts) + 1) * 4), range_of(order, pairs * 4), range_of(slots, pairs * 4),
                          range_of(ws, static_cast<int64_t>(need))};
    st = check_alias(&in, 1, out, 4);
    if (st != QG_OK) return st;
    (void)hipGetLastError();
    launch_sort(sort_params(plan_sort(pairs), ids, pairs, experts, offsets, order, slots, ws), stream);
    return launch_status();
}

int qmoe_route(int dtype, const void *logits, int64_t ld, int64_t rows, int experts, int top, int renorm, int32_t *ids, float *weights,
               int32_t *offsets, int32_t *order, int32_t *slots, void *ws, size_t ws_bytes, hipStream_t stream)
{
    if (!logits || !weights) return QG_ERR_NULL;
    if (!known_dtype(dtype)) return QG_ERR_FORMAT;
    size_t need = 0;
    int st = check_plan(ids, rows, experts, top, offsets, order, slots, ws, ws_bytes, need);
    if (st != QG_OK) return st;
    if (ld < experts || ld > (int64_t(1) << 40) || (renorm != 0 && renorm != 1) || ceil_div(rows, qg::kRouteRows) > kMaxWorkgroups)
        return QG_ERR_SHAPE;
    const int64_t size = dtype == QG_F32 ? 4 : 2, pairs = rows * top;
    if (!aligned(logits, size) || !aligned(weights, 4)) return QG_ERR_ALIGN;
    const Range in = range_of(logits, rows ? ((rows - 1) * ld + experts) * size : 0);
    const Range out[6] = {range_of(offsets, (int64_t(experts) + 1) * 4), range_of(order, pairs * 4), range_of(slots, pairs * 4),
                          range_of(ws, static_cast<int64_t>(need)), range_of(ids, pairs * 4), range_of(weights, pairs * 4)};
    st = check_alias(&in, 1, out, 6);
    if (st != QG_OK) return st;

    (void)hipGetLastError();
    const qg::RouteParams p{logits, ld, rows, experts, top, renorm != 0, ids, weights};
    const qg::SortParams sort = sort_params(plan_sort(pairs), ids, pairs, experts, offsets, order, slots, ws);
    dtype == QG_F32 ? launch_route<float>(p, sort, stream) : launch_route<uint16_t>(p, sort, stream);
    return launch_status();
}

int qmoe_combine(int dtype, const void *y, const int32_t *slots, const float *weights, int64_t rows, int top, int64_t M, int out_dtype,
                 void *out, hipStream_t stream)
{
    if (!y || !slots || !weights || !out) return QG_ERR_NULL;
    if (!known_dtype(dtype) || !known_dtype(out_dtype)) return QG_ERR_FORMAT;
    if (rows < 0 || top < 1 || top > QMOE_MAX_TOP || rows > 0x7fffffffLL / top || M < 1 || M > QMX_MAX_M) return QG_ERR_SHAPE;
    if (!aligned(y, kAlign) || !aligned(out, kAlign) || !aligned(slots, 4) || !aligned(weights, 4)) return QG_ERR_ALIGN;
    if (rows == 0) return QG_OK;
    const int64_t pairs = rows * top, isize = dtype == QG_F32 ? 4 : 2, osize = out_dtype == QG_F32 ? 4 : 2;
    const Range in[3] = {range_of(y, pairs * M * isize), range_of(slots, pairs * 4), range_of(weights, pairs * 4)};
    const Range to = range_of(out, rows * M * osize);
    const int st = check_alias(in, 3, &to, 1);
    if (st != QG_OK) return st;

    (void)hipGetLastError();
    const int64_t per_row = ceil_div(M, 8), step = std::max<int64_t>(1, (int64_t(1) << 30) / per_row);
    for (int64_t first = 0; first < rows; first += step) {
        const int64_t n = std::min(step, rows - first);
        qg::CombineParams p{};
        p.y = y;
        p.slots = slots + first * top;
        p.weights = weights + first * top;
        p.out = static_cast<char *>(out) + first * M * osize;
        p.M = M;
        p.pairs = pairs;
        p.top = top;
        p.pieces = static_cast<uint32_t>(n * per_row);
        p.per_row = qg::fast_div(static_cast<uint32_t>(per_row));
        const dim3 grid(static_cast<unsigned>(ceil_div(p.pieces, qg::kCombineThreads)));
        const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(qg::kCombineThreads), 0, stream, p); };
        const auto pick = [&](auto in_type, auto out_type) {
            using TI = decltype(in_type);
            using TO = decltype(out_type);
            M % 8 == 0 ? go(qg::combine_kernel<TI, TO, true>) : go(qg::combine_kernel<TI, TO, false>);
        };
        if (dtype == QG_F32)
            out_dtype == QG_F32 ? pick(float{}, float{}) : pick(float{}, uint16_t{});
        else
            out_dtype == QG_F32 ? pick(uint16_t{}, float{}) : pick(uint16_t{}, uint16_t{});
    }
    return launch_status();
}

}  // extern "C"
