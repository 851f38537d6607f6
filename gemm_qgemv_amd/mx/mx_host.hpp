// mx_host.hpp -- host-side checks shared by the MX entry points.
#pragma once

#include <atomic>

#include "../serve/host_rows.hpp"
#include "mx_common.hpp"

namespace {

[[maybe_unused]] bool known_dtype(int dtype) { return dtype == QG_F32 || dtype == QG_BF16; }
[[maybe_unused]] bool known_mx(int fmt) { return fmt == QMX_E2M1 || fmt == QMX_E4M3; }

// Inputs of a row: whole blocks, and offsets within a tile of rows fit 32 bits.
[[maybe_unused]] bool mx_k_ok(int64_t k) { return k >= 32 && k % 32 == 0 && k <= QMX_MAX_K; }

[[maybe_unused]] int64_t mx_row_bytes(int fmt, int64_t k) { return fmt == QMX_E2M1 ? k / 2 : k; }

// Tokens, experts and experts a token: their pairs are counted in 32 bits.
[[maybe_unused]] bool moe_sizes_ok(int64_t rows, int experts, int top)
{
    return rows >= 0 && experts >= 1 && experts <= QMOE_MAX_EXPERTS && top >= 1 && top <= QMOE_MAX_TOP && top <= experts &&
           rows <= 0x7fffffffLL / top;
}

// Lets a kernel be launched with up to `bytes` of dynamic LDS: asked for on
// its first call on a device, which `asked` remembers (where it is refused, so is
// the launch).
[[maybe_unused]] void allow_dynamic_lds(const void *kernel, size_t bytes, std::atomic<uint64_t> &asked)
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (asked.load(std::memory_order_relaxed) & bit) return;
    if (hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) == hipSuccess)
        asked.fetch_or(bit, std::memory_order_relaxed);
}

}  // namespace
