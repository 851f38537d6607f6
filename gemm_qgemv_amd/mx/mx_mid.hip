// mx_mid.hip -- launches of the MX products for some tens of rows.
#include "mx_call.hpp"
#include "mx_mid.hpp"

namespace qg {

namespace {

template <typename F, int MI, int NJ>
void launch(const MxCall &c, MxGemmParams p, hipStream_t stream)
{
    p.tiles_m = static_cast<int>(ceil_div(c.M, 32 * MI / (F::SILU ? 2 : 1)));
    p.tiles_n = static_cast<int>(c.row_tiles(16 * NJ));
    static std::atomic<uint64_t> asked{0};
    constexpr size_t bytes = MxMidLds<F::XF, MI, NJ>::bytes;
    const auto kernel = &mx_mid_kernel<F::XF, typename F::T, F::SILU, F::GROUPED, MI, NJ>;
    allow_dynamic_lds(reinterpret_cast<const void *>(kernel), bytes, asked);
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(int64_t(p.tiles_m) * p.tiles_n)), dim3(kMidThreads), bytes, stream, p);
}

}  // namespace

void mx_launch_mid(const MxCall &c, const MxGemmParams &p, int mi, int nj, hipStream_t stream)
{
    mx_dispatch(c, [&](auto form) {
        using F = decltype(form);
        const auto rows = [&](auto blocks) {
            constexpr int MI = decltype(blocks)::value;
            switch (nj) {
                case 2: return launch<F, MI, 2>(c, p, stream);
                case 4: return launch<F, MI, 4>(c, p, stream);
                case 6: return launch<F, MI, 6>(c, p, stream);
                default: return launch<F, MI, 8>(c, p, stream);
            }
        };
        mi == 4 ? rows(std::integral_constant<int, 4>{}) : rows(std::integral_constant<int, 2>{});
    });
}

}  // namespace qg
