// mx_few.hip -- launches of the MX products for few rows.
#include "mx_call.hpp"
#include "mx_few.hpp"

namespace qg {

void mx_launch_few(const MxCall &c, const MxGemmParams &from, bool side_by_side, hipStream_t stream)
{
    const auto go = [&](auto kernel, int outputs) {
        MxGemmParams p = from;
        p.tiles_m = static_cast<int>(ceil_div(c.M, outputs));
        p.tiles_n = static_cast<int>(c.row_tiles(16));
        hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(int64_t(p.tiles_m) * p.tiles_n)), dim3(kFewThreads), 0, stream, p);
    };
    mx_dispatch(c, [&](auto form) {
        using F = decltype(form);
        constexpr int MI = F::SILU ? 1 : 2;
        if (side_by_side)
            go(mx_few_kernel<F::XF, typename F::T, F::SILU, F::GROUPED, MI, 1>, 16 * MI * kFewWaves);
        else
            go(mx_few_kernel<F::XF, typename F::T, F::SILU, F::GROUPED, 1, kFewWaves>, 16);
    });
}

}  // namespace qg
