// host_args.hpp -- argument checks shared by the library's entry points
// (host only; they run before anything is enqueued).
#pragma once

#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include "../../include/qg.h"

namespace {

constexpr int64_t kAlign = 16;
// Compute units of the MI355X.
constexpr int64_t kComputeUnits = 256;

[[maybe_unused]] bool aligned(const void *p, int64_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

[[maybe_unused]] int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
[[maybe_unused]] int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
[[maybe_unused]] size_t align256(size_t n) { return (n + 255) / 256 * 256; }

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};

[[maybe_unused]] Range range_of(const void *p, int64_t bytes)
{
    uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{a, a + static_cast<uintptr_t>(bytes)};
}

[[maybe_unused]] bool overlap(Range a, Range b)
{
    return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo;
}

// Every written range must be disjoint from every input range and from
// every other written range (an exact alias such as y == x is an overlap
// like any other).
[[maybe_unused]] int check_alias(const Range *inputs, int n_inputs, const Range *written, int n_written)
{
    for (int i = 0; i < n_written; ++i)
        for (int j = 0; j < n_inputs; ++j)
            if (overlap(written[i], inputs[j])) return QG_ERR_ALIAS;
    for (int i = 0; i < n_written; ++i)
        for (int j = i + 1; j < n_written; ++j)
            if (overlap(written[i], written[j])) return QG_ERR_ALIAS;
    return QG_OK;
}

[[maybe_unused]] int launch_status()
{
    hipError_t e = hipGetLastError();
    return e == hipSuccess ? QG_OK : QG_ERR_LAUNCH;
}

}  // namespace
