// quant.hpp -- rows quantized into MX blocks, and the values MX rows stand for.
//
// A block's scale is the power of two of its largest magnitude, less the
// element type's largest exponent (OCP Microscaling Formats 1.0, section 6.3);
// elements are rounded to nearest even at that scale, and what lies beyond the
// largest element becomes it. With E the exponent field of the largest
// magnitude the scale byte is max(E - emax, 0), subnormal blocks included, so
// the whole quantizer is exact arithmetic and one rounding.
//
// A lane holds 8 elements, 4 lanes a block, 16 lanes 128 elements, whose four
// scale bytes they store as one dword. Bound by HBM: 16411 x 6144 bf16 to e2m1 61 us
// (4.2 TB/s of 5.16 that a copy reaches), back to float32 98 us (4.6 TB/s); 64 x
// 2048 2.3 us a launch, all of it latency.
#pragma once

#include "mx_common.hpp"

namespace qg {

constexpr int kQuantThreads = 256;
constexpr int kQuantUnit = 128;      // elements that 16 lanes take

struct QuantParams {
    const void *x;
    int64_t stride;       // elements between rows of x
    uint8_t *codes, *scales;
    uint32_t units;       // 16-lane units: rows * per_row
    int32_t k;            // elements of a row
    FastDiv per_row;      // units of a row
};

// 8 elements at a scale of 2^(byte - 127) as 4 or 8 bytes of codes.
template <int FMT>
__device__ __forceinline__ uint2 mx_codes(const float (&x)[8], uint32_t byte)
{
    const float scale = __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
    uint2 out = make_uint2(0, 0);
    if constexpr (FMT == kMxE2M1) {
        // rounds to nearest even and takes what is beyond 6 as 6
        out.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out.x, x[0], x[1], scale, 0);
        out.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out.x, x[2], x[3], scale, 1);
        out.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out.x, x[4], x[5], scale, 2);
        out.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out.x, x[6], x[7], scale, 3);
    } else {
        // the conversion makes what is beyond 448 a NaN, so that is cut first
        // (448 * 2^(byte - 127) is a normal float32: byte <= 246)
        const float top = 448.0f * scale;
        float c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = __builtin_amdgcn_fmed3f(x[i], -top, top);
        typedef short s16x2 __attribute__((ext_vector_type(2)));
        s16x2 a = {0, 0}, b = {0, 0};
        a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, c[0], c[1], scale, false);
        a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, c[2], c[3], scale, true);
        b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, c[4], c[5], scale, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, c[6], c[7], scale, true);
        out.x = __builtin_bit_cast(uint32_t, a);
        out.y = __builtin_bit_cast(uint32_t, b);
    }
    return out;
}

template <typename T, int FMT>
__global__ __launch_bounds__(kQuantThreads) void mx_quant_kernel(QuantParams p)
{
    const uint32_t unit = blockIdx.x * (kQuantThreads / 16) + (threadIdx.x >> 4);
    if (unit >= p.units) return;                       // 16 lanes leave together
    const uint32_t row = unit / p.per_row, part = unit - row * p.per_row.d;
    const int lane = threadIdx.x & 15;
    const int k = part * kQuantUnit + lane * 8;
    const bool in = k < p.k;                           // whole blocks: k is a multiple of 32
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.0f;
    if (in) load8(static_cast<const T *>(p.x) + int64_t(row) * p.stride + k, x);
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) big = max(big, __float_as_uint(x[i]) & 0x7fffffffu);
    big = max(big, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(big), 0xB1, 0xF, 0xF, false)));   // lane ^ 1
    big = max(big, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(big), 0x4E, 0xF, 0xF, false)));   // lane ^ 2
    const int e = static_cast<int>(big >> 23);         // 255: an infinity or a NaN in the block
    uint32_t byte = static_cast<uint32_t>(max(e - kMxEmax<FMT>, 0));
    uint2 codes = mx_codes<FMT>(x, byte);
    if (e == 255) byte = 255, codes = make_uint2(0, 0);
    const int64_t at = int64_t(row) * mx_bytes<FMT>(p.k) + mx_bytes<FMT>(k);
    if (in) {
        if constexpr (FMT == kMxE2M1)
            *reinterpret_cast<uint32_t *>(p.codes + at) = codes.x;
        else
            *reinterpret_cast<uint2 *>(p.codes + at) = codes;
    }
    // the four quads' bytes side by side (0 behind the row's end)
    int four = static_cast<int>((in ? byte : 0) << (8 * (lane >> 2)));
    four |= __builtin_amdgcn_update_dpp(0, four, 0x124, 0xF, 0xF, false);     // rotated by 4 lanes of 16
    four |= __builtin_amdgcn_update_dpp(0, four, 0x128, 0xF, 0xF, false);     // by 8
    if (lane == 0) *reinterpret_cast<int *>(p.scales + int64_t(row) * mx_pitch(p.k) + part * 4) = four;
}

struct DequantParams {
    const uint8_t *codes, *scales;
    void *x;
    int64_t stride;
    uint32_t units;
    int32_t k;
    FastDiv per_row;
};

template <typename T, int FMT>
__global__ __launch_bounds__(kQuantThreads) void mx_dequant_kernel(DequantParams p)
{
    const uint32_t unit = blockIdx.x * (kQuantThreads / 16) + (threadIdx.x >> 4);
    if (unit >= p.units) return;
    const uint32_t row = unit / p.per_row, part = unit - row * p.per_row.d;
    const int k = part * kQuantUnit + (threadIdx.x & 15) * 8;
    if (k >= p.k) return;
    const uint8_t *src = p.codes + int64_t(row) * mx_bytes<FMT>(p.k) + mx_bytes<FMT>(k);
    const uint32_t byte = p.scales[int64_t(row) * mx_pitch(p.k) + k / kMxBlock];
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    f32x2 v[4];
    if constexpr (FMT == kMxE2M1) {
        const uint32_t c = *reinterpret_cast<const uint32_t *>(src);
        v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
        v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
        v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
        v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
    } else {
        const uint2 c = *reinterpret_cast<const uint2 *>(src);
        v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.x, 1.0f, false);
        v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.x, 1.0f, true);
        v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.y, 1.0f, false);
        v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.y, 1.0f, true);
    }
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // exact, subnormal results too
        x[i] = __builtin_ldexpf(v[i / 2][i % 2], static_cast<int>(byte) - 127);
        if (byte == 255) x[i] = __builtin_nanf("");
    }
    store8(static_cast<T *>(p.x) + int64_t(row) * p.stride + k, x);
}

}  // namespace qg
