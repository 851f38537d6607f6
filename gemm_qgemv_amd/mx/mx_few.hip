// mx_few.hip -- launches of the MX products for few rows.
#include "mx_call.hpp"
#include "mx_few.hpp"

namespace qg {

void mx_launch_few(const MxCall &c, const MxGemmParams &from, int blocks, int waves, hipStream_t stream)
{
    const auto go = [&](auto kernel, int outputs) {
        MxGemmParams p = from;
        p.tiles_m = static_cast<int>(ceil_div(c.M, outputs));
        p.tiles_n = static_cast<int>(c.row_tiles(16));
        hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(int64_t(p.tiles_m) * p.tiles_n)), dim3(kFewThreads), 0, stream, p);
    };
    mx_dispatch(c, [&](auto form) {
        using F = decltype(form);
        const auto split = [&](auto mi) {
            constexpr int MI = decltype(mi)::value, EACH = 16 * MI * kFewWaves;
            if (waves == 4)
                go(mx_few_kernel<F::XF, typename F::T, F::SILU, F::GROUPED, MI, 4>, EACH / 4);
            else if (waves == 2)
                go(mx_few_kernel<F::XF, typename F::T, F::SILU, F::GROUPED, MI, 2>, EACH / 2);
            else
                go(mx_few_kernel<F::XF, typename F::T, F::SILU, F::GROUPED, MI, 1>, EACH);
        };
        if constexpr (F::SILU)
            split(std::integral_constant<int, 1>{});
        else
            blocks == 2 ? split(std::integral_constant<int, 2>{}) : split(std::integral_constant<int, 1>{});
    });
}

}  // namespace qg
