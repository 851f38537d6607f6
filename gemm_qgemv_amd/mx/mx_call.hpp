// mx_call.hpp -- an MX product as the host sees it, shared by the files that
// hold its kernels (host only).
#pragma once

#include <algorithm>
#include <type_traits>

#include "mx_gemm.hpp"
#include "mx_host.hpp"

namespace qg {

struct MxCall {
    int xfmt, act, dtype;
    bool grouped;
    int64_t M, K, N;        // N: rows, or pairs of the grouped form
    int experts;

    // Rows of weights (of one expert), gate and up both.
    int64_t wide() const { return M * (act == QMX_SILU_MUL ? 2 : 1); }

    // Tiles of T rows: of all rows, or at most of the experts' rows (each of the
    // experts that has rows leaves one tile part empty).
    int64_t row_tiles(int64_t T) const
    {
        if (!grouped) return (N + T - 1) / T;
        const int64_t some = std::min<int64_t>(experts, N);
        return std::min(N, (N + some * (T - 1)) / T);
    }
};

template <int XF_, typename T_, bool SILU_, bool GROUPED_>
struct MxForm {
    static constexpr int XF = XF_;
    using T = T_;
    static constexpr bool SILU = SILU_, GROUPED = GROUPED_;
};

// f(MxForm of the call).
template <typename F>
void mx_dispatch(const MxCall &c, F f)
{
    const auto typed = [&](auto xf, auto type) {
        constexpr int XF = decltype(xf)::value;
        using T = decltype(type);
        if (c.act == QMX_SILU_MUL)
            c.grouped ? f(MxForm<XF, T, true, true>{}) : f(MxForm<XF, T, true, false>{});
        else
            c.grouped ? f(MxForm<XF, T, false, true>{}) : f(MxForm<XF, T, false, false>{});
    };
    const auto kind = [&](auto xf) { c.dtype == QG_F32 ? typed(xf, float{}) : typed(xf, uint16_t{}); };
    if (c.xfmt == QMX_E2M1)
        kind(std::integral_constant<int, kMxE2M1>{});
    else
        kind(std::integral_constant<int, kMxE4M3>{});
}

// The launches of each kernel's file.
// blocks: of 16 outputs a wave takes (1 with SILU), waves: that split K
void mx_launch_few(const MxCall &c, const MxGemmParams &p, int blocks, int waves, hipStream_t stream);
// mi: blocks of 16 weight rows a wave takes (2 or 4), nj: blocks of 16 rows of x (2, 4,
// and 6, or where mi is 4 mx_mid_most: more would not fit in registers)
constexpr int mx_mid_most(int xfmt) { return xfmt == QMX_E2M1 ? 6 : 5; }
void mx_launch_mid(const MxCall &c, const MxGemmParams &p, int mi, int nj, hipStream_t stream);
// size: 64, 128 (of e2m1 rows only) or 256, the tile's weight rows
void mx_launch_tile(const MxCall &c, const MxGemmParams &p, int size, void *ws, hipStream_t stream);

// Rows of x in a tile of `size` weight rows, and what its launches need.
int64_t mx_tile_rows(const MxCall &c, int size);
size_t mx_tile_workspace(const MxCall &c, int size);
int64_t mx_tile_workgroups(const MxCall &c, int size);

}  // namespace qg
