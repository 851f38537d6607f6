// host_rows.hpp -- what the serving-step entry points share beside
// host_args.hpp: how large a grid may be, and rows that lie apart.
#pragma once

#include "../csrc/host_args.hpp"

namespace {

// Workgroups of 256 threads in one dimension of a launch: it has fewer than 2^32
// threads. (A larger grid is not reported as an error; part of it is not run.)
[[maybe_unused]] constexpr int64_t kMaxWorkgroups = (int64_t(1) << 24) - 1;

// n rows of `width` bytes, `stride` bytes apart.
struct Rows {
    uintptr_t lo;
    int64_t n, stride, width;
};

// Whether rows of two buffers share bytes. Rows as far apart in both may be parts
// of the same wider rows; else a buffer counts from its first to its last byte.
[[maybe_unused]] bool overlap(const Rows &a, const Rows &b)
{
    const auto end = [](const Rows &r) { return r.lo + static_cast<uintptr_t>((r.n - 1) * r.stride + r.width); };
    if (!overlap(Range{a.lo, end(a)}, Range{b.lo, end(b)})) return false;
    if (a.stride != b.stride) return true;
    const bool up = b.lo >= a.lo;
    const int64_t by = static_cast<int64_t>((up ? b.lo - a.lo : a.lo - b.lo) % static_cast<uintptr_t>(a.stride));
    return by < (up ? a : b).width || by + (up ? b : a).width > a.stride;
}

}  // namespace
