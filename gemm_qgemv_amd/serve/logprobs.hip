// logprobs.hip -- entry point of the token log probabilities: checks, the
// cut of rows into slices, launches.
#include "host_rows.hpp"

#include <algorithm>

#include "logprobs.hpp"

namespace {

struct LogprobPlan {
    int nslice;
    int32_t slice;
};

// Rows are cut until there are four workgroups a compute unit, but not into
// less than one block a wave.
LogprobPlan plan_logprobs(int64_t rows, int64_t vocab)
{
    const int64_t unit = qg::kLpBlock * qg::kLpWaves;
    const int64_t span = vocab + 3;                       // with the row's distance from its 16-byte boundary
    const int64_t want = std::clamp<int64_t>(ceil_div(4 * kComputeUnits, rows), 1, ceil_div(span, unit));
    LogprobPlan a;
    a.slice = static_cast<int32_t>(round_up(ceil_div(span, want), unit));
    a.nslice = static_cast<int>(ceil_div(span, a.slice));
    return a;
}

size_t stat_bytes(const LogprobPlan &a, int64_t rows) { return align256(static_cast<size_t>(rows) * a.nslice * 16); }

size_t logprob_workspace(const LogprobPlan &a, int64_t rows, int top)
{
    return a.nslice == 1 ? 0 : stat_bytes(a, rows) + align256(static_cast<size_t>(rows) * a.nslice * top * 8);
}

bool logprob_sizes_ok(int64_t rows, int64_t vocab, int top)
{
    return rows >= 1 && rows <= 0x7fffffffLL && vocab >= 1 && vocab <= (int64_t(1) << 30) && top >= 0 &&
           top <= QG_MAX_TOP && top <= vocab && rows * plan_logprobs(rows, vocab).nslice <= 0x7fffffffLL;
}

}  // namespace

extern "C" {

size_t qlogprobs_workspace_bytes(int64_t rows, int64_t vocab, int top)
{
    return logprob_sizes_ok(rows, vocab, top) ? logprob_workspace(plan_logprobs(rows, vocab), rows, top) : 0;
}

int qlogprobs(const float *logits, int64_t ld, int64_t rows, int64_t vocab, const int32_t *ids, int top,
              float *logprob, float *entropy, int32_t *rank, int32_t *top_ids, float *top_logprobs,
              void *ws, size_t ws_bytes, hipStream_t stream)
{
    if (!logits) return QG_ERR_NULL;
    if (!logprob_sizes_ok(rows, vocab, top) || ld < vocab || ld > (int64_t(1) << 40)) return QG_ERR_SHAPE;
    if ((!ids && (logprob || rank)) || (top > 0) != (top_ids != nullptr) || (top > 0) != (top_logprobs != nullptr))
        return QG_ERR_NULL;
    for (const void *p : {static_cast<const void *>(logits), static_cast<const void *>(ids), static_cast<const void *>(logprob),
                          static_cast<const void *>(entropy), static_cast<const void *>(rank),
                          static_cast<const void *>(top_ids), static_cast<const void *>(top_logprobs)})
        if (!aligned(p, 4)) return QG_ERR_ALIGN;
    const LogprobPlan a = plan_logprobs(rows, vocab);
    const size_t need = logprob_workspace(a, rows, top);
    if (need > 0) {
        if (!ws || ws_bytes < need) return QG_ERR_WORKSPACE;
        if (!aligned(ws, kAlign)) return QG_ERR_ALIGN;
    }
    Range inputs[2] = {range_of(logits, ((rows - 1) * ld + vocab) * 4), range_of(ids, ids ? rows * 4 : 0)};
    Range written[6] = {range_of(logprob, logprob ? rows * 4 : 0),
                        range_of(entropy, entropy ? rows * 4 : 0),
                        range_of(rank, rank ? rows * 4 : 0),
                        range_of(top_ids, rows * top * 4),
                        range_of(top_logprobs, rows * top * 4),
                        range_of(ws, static_cast<int64_t>(need))};
    const int st = check_alias(inputs, 2, written, 6);
    if (st != QG_OK) return st;

    (void)hipGetLastError();
    qg::LogprobParams p{};
    p.ld = ld;
    p.vocab = static_cast<int32_t>(vocab);
    p.top = top;
    p.nslice = a.nslice;
    p.slice = a.slice;
    if (a.nslice > 1) {
        p.part = static_cast<qg::f32x4 *>(ws);
        p.part_keys = reinterpret_cast<uint64_t *>(static_cast<char *>(ws) + stat_bytes(a, rows));
    }
    // in pieces that a grid holds (rows are cut into slices only where they are few)
    for (int64_t first = 0; first < rows; first += p.rows) {
        p.rows = a.nslice > 1 ? rows : std::min(rows - first, kMaxWorkgroups);
        p.x = logits + first * ld;
        auto at = [&](auto *base, int64_t step) { return base ? base + first * step : nullptr; };
        p.ids = at(ids, 1);
        p.logprob = at(logprob, 1);
        p.entropy = at(entropy, 1);
        p.rank = at(rank, 1);
        p.top_ids = at(top_ids, top);
        p.top_logprobs = at(top_logprobs, top);
        hipLaunchKernelGGL(qg::logprob_kernel, dim3(static_cast<unsigned>(p.rows * a.nslice)), dim3(qg::kLpThreads), 0, stream, p);
    }
    if (a.nslice > 1)
        hipLaunchKernelGGL(qg::logprob_join_kernel, dim3(static_cast<unsigned>(rows)), dim3(qg::kLpJoinThreads), 0, stream, p);
    return launch_status();
}

}  // extern "C"
