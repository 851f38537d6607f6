// quant.hip -- entry points of the MX quantizer: checks, launches.
#include "mx_host.hpp"
#include "quant.hpp"

#include <algorithm>

namespace {

// Launches of at most this many units: a grid holds them, and their numbers
// are below 2^31.
constexpr int64_t kMaxUnits = int64_t(1) << 27;

int check_rows(int dtype, const void *x, int64_t stride, int64_t rows, int64_t k, int fmt, const void *codes, const void *scales)
{
    if (!x || !codes || !scales) return QG_ERR_NULL;
    if (!known_dtype(dtype) || !known_mx(fmt)) return QG_ERR_FORMAT;
    const int64_t size = dtype == QG_F32 ? 4 : 2;
    if (!mx_k_ok(k) || rows < 0 || rows > 0x7fffffffLL || stride < k || stride > (int64_t(1) << 40) || stride * size % kAlign != 0)
        return QG_ERR_SHAPE;
    if (!aligned(x, kAlign) || !aligned(codes, kAlign) || !aligned(scales, 4)) return QG_ERR_ALIGN;
    return QG_OK;
}

}  // namespace

extern "C" {

int64_t qmx_scale_pitch(int64_t K) { return mx_k_ok(K) ? qg::mx_pitch(K) : 0; }

int qmx_quant(int dtype, const void *x, int64_t x_stride, int64_t rows, int64_t K, int fmt, void *codes, void *scales,
              hipStream_t stream)
{
    int st = check_rows(dtype, x, x_stride, rows, K, fmt, codes, scales);
    if (st != QG_OK || rows == 0) return st;
    const int64_t size = dtype == QG_F32 ? 4 : 2;
    const Range in = range_of(x, ((rows - 1) * x_stride + K) * size);
    const Range out[2] = {range_of(codes, rows * mx_row_bytes(fmt, K)), range_of(scales, rows * qg::mx_pitch(K))};
    st = check_alias(&in, 1, out, 2);
    if (st != QG_OK) return st;

    (void)hipGetLastError();
    const int64_t per_row = ceil_div(K, qg::kQuantUnit), step = std::max<int64_t>(1, kMaxUnits / per_row);
    for (int64_t first = 0; first < rows; first += step) {
        const int64_t n = std::min(step, rows - first);
        qg::QuantParams p{};
        p.x = static_cast<const char *>(x) + first * x_stride * size;
        p.stride = x_stride;
        p.codes = static_cast<uint8_t *>(codes) + first * mx_row_bytes(fmt, K);
        p.scales = static_cast<uint8_t *>(scales) + first * qg::mx_pitch(K);
        p.units = static_cast<uint32_t>(n * per_row);
        p.k = static_cast<int32_t>(K);
        p.per_row = qg::fast_div(static_cast<uint32_t>(per_row));
        const dim3 grid(static_cast<unsigned>(ceil_div(p.units, qg::kQuantThreads / 16)));
        const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(qg::kQuantThreads), 0, stream, p); };
        if (dtype == QG_F32)
            fmt == QMX_E2M1 ? go(qg::mx_quant_kernel<float, qg::kMxE2M1>) : go(qg::mx_quant_kernel<float, qg::kMxE4M3>);
        else
            fmt == QMX_E2M1 ? go(qg::mx_quant_kernel<uint16_t, qg::kMxE2M1>) : go(qg::mx_quant_kernel<uint16_t, qg::kMxE4M3>);
    }
    return launch_status();
}

int qmx_dequant(int fmt, const void *codes, const void *scales, int64_t rows, int64_t K, int dtype, void *x, int64_t x_stride,
                hipStream_t stream)
{
    int st = check_rows(dtype, x, x_stride, rows, K, fmt, codes, scales);
    if (st != QG_OK || rows == 0) return st;
    const int64_t size = dtype == QG_F32 ? 4 : 2;
    const Range in[2] = {range_of(codes, rows * mx_row_bytes(fmt, K)), range_of(scales, rows * qg::mx_pitch(K))};
    const Range out = range_of(x, ((rows - 1) * x_stride + K) * size);
    st = check_alias(in, 2, &out, 1);
    if (st != QG_OK) return st;

    (void)hipGetLastError();
    const int64_t per_row = ceil_div(K, qg::kQuantUnit), step = std::max<int64_t>(1, kMaxUnits / per_row);
    for (int64_t first = 0; first < rows; first += step) {
        const int64_t n = std::min(step, rows - first);
        qg::DequantParams p{};
        p.codes = static_cast<const uint8_t *>(codes) + first * mx_row_bytes(fmt, K);
        p.scales = static_cast<const uint8_t *>(scales) + first * qg::mx_pitch(K);
        p.x = static_cast<char *>(x) + first * x_stride * size;
        p.stride = x_stride;
        p.units = static_cast<uint32_t>(n * per_row);
        p.k = static_cast<int32_t>(K);
        p.per_row = qg::fast_div(static_cast<uint32_t>(per_row));
        const dim3 grid(static_cast<unsigned>(ceil_div(p.units, qg::kQuantThreads / 16)));
        const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(qg::kQuantThreads), 0, stream, p); };
        if (dtype == QG_F32)
            fmt == QMX_E2M1 ? go(qg::mx_dequant_kernel<float, qg::kMxE2M1>) : go(qg::mx_dequant_kernel<float, qg::kMxE4M3>);
        else
            fmt == QMX_E2M1 ? go(qg::mx_dequant_kernel<uint16_t, qg::kMxE2M1>) : go(qg::mx_dequant_kernel<uint16_t, qg::kMxE4M3>);
    }
    return launch_status();
}

}  // extern "C"
