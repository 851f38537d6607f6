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
        constexpr int most = mx_mid_most(F::XF == kMxE2M1 ? QMX_E2M1 : QMX_E4M3);
        switch (nj) {
            case 2: return mi == 4 ? launch<F, 4, 2>(c, p, stream) : launch<F, 2, 2>(c, p, stream);
            case 4: return mi == 4 ? launch<F, 4, 4>(c, p, stream) : launch<F, 2, 4>(c, p, stream);
            default: return mi == 4 ? launch<F, 4, most>(c, p, stream) : launch<F, 2, 6>(c, p, stream);
        }
    });
}

}  // namespace qg
