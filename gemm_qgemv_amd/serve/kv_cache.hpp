// kv_cache.hpp -- the paged 4-bit key/value cache as the kernels see it, and
// the element types of activations.
//
// One page of one key/value head is one block of bytes (include/qg.h): K
// codes [page][D/2], K coefficients [page][D/64][2] (bf16 scale, bias), then
// the same two parts for V. A token's codes and its coefficients are each
// contiguous, so a tile of tokens is read in 16-byte pieces of whole rows,
// and a page moves as one piece.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../csrc/qg_device.hpp"

namespace qg {

struct KvView {
    uint8_t *data;
    int64_t page_bytes;    // of all heads
    int32_t num_pages;
    int32_t block_bytes;   // of one head
    int32_t page_shift;    // log2(page_size)
    int32_t heads, dim;
    int32_t dim_shift;     // log2(head_dim)
};

__host__ __device__ constexpr int kv_coef_bytes(int dim) { return dim / 16; }   // of one token, K or V

// Byte offset in a block of the codes of K (part 0) or V (part 1), and of
// the coefficients behind them.
__device__ __forceinline__ int kv_part(const KvView &c, int part) { return part * (c.block_bytes >> 1); }
__device__ __forceinline__ int kv_coefs(const KvView &c, int part)
{
    return kv_part(c, part) + ((c.dim / 2) << c.page_shift);
}

// float32 -> bf16 bits, nearest even (gfx950 converts; NaN stays NaN).
__device__ __forceinline__ uint32_t f32_to_bf16_bits(float v)
{
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// Two of them, the first in the low half.
__device__ __forceinline__ uint32_t f32_to_bf16_pair(float a, float b)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
    return __builtin_bit_cast(uint32_t, v);
}

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Eight consecutive activations (16-byte aligned) as float32.
template <typename T>
__device__ __forceinline__ void load8(const T *src, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float *src, float (&x)[8])
{
    const f32x4 a = reinterpret_cast<const f32x4 *>(src)[0], b = reinterpret_cast<const f32x4 *>(src)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
}
template <>
__device__ __forceinline__ void load8<uint16_t>(const uint16_t *src, float (&x)[8])
{
    const u32x4 a = *reinterpret_cast<const u32x4 *>(src);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(a[i] << 16);
        x[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
}

template <typename T>
__device__ __forceinline__ void store8(T *dst, const float (&x)[8]);
template <>
__device__ __forceinline__ void store8<float>(float *dst, const float (&x)[8])
{
    reinterpret_cast<f32x4 *>(dst)[0] = f32x4{x[0], x[1], x[2], x[3]};
    reinterpret_cast<f32x4 *>(dst)[1] = f32x4{x[4], x[5], x[6], x[7]};
}
template <>
__device__ __forceinline__ void store8<uint16_t>(uint16_t *dst, const float (&x)[8])
{
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f32_to_bf16_pair(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<u32x4 *>(dst) = v;
}

}  // namespace qg
