// kv_host.hpp -- host-side checks of the key/value cache's description,
// shared by the entry points that take one.
#pragma once

#include <atomic>

#include "host_rows.hpp"
#include "kv_cache.hpp"

namespace {

[[maybe_unused]] bool known_dtype(int dtype) { return dtype == QG_F32 || dtype == QG_BF16; }

[[maybe_unused]] int check_geometry(const qg_kv_cache &c)
{
    const bool page_ok = c.page_size >= 16 && c.page_size <= 256 && (c.page_size & (c.page_size - 1)) == 0;
    if (!page_ok || c.num_pages < 1 || c.num_pages > 0x7fffffffLL / c.page_size || c.kv_heads < 1 ||
        c.kv_heads > 1024 || (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256))
        return QG_ERR_SHAPE;
    return QG_OK;
}

// Bytes of one page of one head.
[[maybe_unused]] int64_t block_bytes(const qg_kv_cache &c)
{
    return int64_t(c.page_size) * (c.head_dim + c.head_dim / 8);
}

[[maybe_unused]] int64_t cache_bytes(const qg_kv_cache &c) { return c.num_pages * c.kv_heads * block_bytes(c); }

[[maybe_unused]] int check_cache(const qg_kv_cache &c)
{
    const int st = check_geometry(c);
    if (st != QG_OK) return st;
    return aligned(c.data, kAlign) ? QG_OK : QG_ERR_ALIGN;
}

[[maybe_unused]] qg::KvView kv_view(const qg_kv_cache &c)
{
    qg::KvView v;
    v.data = static_cast<uint8_t *>(c.data);
    v.num_pages = static_cast<int32_t>(c.num_pages);
    v.block_bytes = static_cast<int32_t>(block_bytes(c));
    v.page_bytes = int64_t(c.kv_heads) * v.block_bytes;
    v.page_shift = __builtin_ctz(static_cast<unsigned>(c.page_size));
    v.heads = c.kv_heads;
    v.dim = c.head_dim;
    v.dim_shift = __builtin_ctz(static_cast<unsigned>(c.head_dim));
    return v;
}

// Lets a kernel be launched with up to `bytes` of dynamic LDS: asked for on
// its first call on a device (where it is refused, so is the launch).
template <auto KERNEL>
[[maybe_unused]] void allow_lds(size_t bytes)
{
    static std::atomic<uint64_t> asked{0};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (asked.load(std::memory_order_relaxed) & bit) return;
    if (hipFuncSetAttribute(reinterpret_cast<const void *>(KERNEL), hipFuncAttributeMaxDynamicSharedMemorySize,
                            static_cast<int>(bytes)) == hipSuccess)
        asked.fetch_or(bit, std::memory_order_relaxed);
}

}  // namespace
