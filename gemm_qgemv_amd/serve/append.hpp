// append.hpp -- keys and values quantized into their slots of the 4-bit
// cache, and the values of slots read back.
//
// A group of 64 channels is held by 8 lanes of 8 values: minimum and maximum
// by DPP over the 8 lanes, scale = bf16((max - min) * (1 / 15)), bias = bf16(min),
// code = round_half_even((x - bias) / scale) into 0..15 (I Built an LLM
// Inference Engine on a 15 year old GPU..., "Quantization: The Model Doesn't
// Run on INT4": the scale is the range over 15, the minimum is kept). A lane
// then stores its 8 codes as one dword: 8 lanes write a group's 32 bytes.
// Bound by HBM at a prompt's sizes, with the vector unit close behind for
// append (16411 tokens of 8 heads of 128 bfloat16 channels: 86 MB in 20 us,
// 4.3 TB/s, vector unit 77% busy; read back as float32 153 MB in 30.7 us, 5.0
// TB/s), by latency at a decode step's (64 tokens 3.1 and 2.7 us).
#pragma once

#include "kv_cache.hpp"

namespace qg {

// How threads map to (token, run of 8 channels): a workgroup takes whole
// rows while they fit, else a piece of one row (blockIdx.z).
struct AppendMap {
    int per_row;      // runs of 8 channels in a row: kv_heads * head_dim / 8
    int rows;         // rows a workgroup takes
    float inv;        // 1 / per_row
};

__device__ __forceinline__ bool append_place(const AppendMap &m, int64_t n, int64_t &t, int &c)
{
    // exact: threadIdx.x < 256, and the quotient is off by less than 1/per_row
    const int row = m.rows > 1 ? static_cast<int>((static_cast<float>(threadIdx.x) + 0.5f) * m.inv) : 0;
    const int run = blockIdx.z * blockDim.x + threadIdx.x - row * m.per_row;
    t = int64_t(blockIdx.x) * m.rows + row;
    c = run * 8;
    return row < m.rows && run < m.per_row && t < n;
}

struct AppendParams {
    const char *src[2];       // k, v
    int64_t stride[2];        // elements between rows
    const int32_t *slots;
    int64_t n;
    AppendMap map;
    KvView kv;
};

constexpr int kAppendThreads = 256;

// Minimum (or maximum) over the 8 lanes of an aligned run of 8.
template <bool MAX>
__device__ __forceinline__ float reduce8(float v)
{
    auto step = [](float a, float b) { return MAX ? fmaxf(a, b) : fminf(a, b); };
    v = step(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false)));   // lane ^ 1
    v = step(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false)));   // lane ^ 2
    // the lane mirrored within its run of 8 (the quads hold one value each now)
    return step(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false)));
}

// The scale is the range times this, one operation where a division takes 10;
// the product is off by at most one bit of 24 before it is rounded to 8.
constexpr float kFifteenth = 1.0f / 15.0f;

// A group of 64 values (8 lanes of 8) as bf16 bits of scale and bias (low and
// high half of `coef`) and this lane's 8 codes.
__device__ __forceinline__ void quantize_group(const float (&x)[8], int lane, uint32_t &codes, uint32_t &coef)
{
    float lo = x[0], hi = x[0];
    uint32_t largest = 0;                         // as bits: not finite from 0x7f800000 on
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        largest = max(largest, __float_as_uint(x[i]) & 0x7fffffffu);
    }
    lo = reduce8<false>(lo);
    hi = reduce8<true>(hi);
    const uint64_t ok = __ballot(largest < 0x7f800000u);
    const uint32_t both = f32_to_bf16_pair((hi - lo) * kFifteenth, lo);
    uint32_t sb = both & 0xffffu, bb = both >> 16;
    const bool good = ((ok >> (lane & 56)) & 0xff) == 0xff && (sb & 0x7f80u) != 0x7f80u && (bb & 0x7f80u) != 0x7f80u;
    if ((sb & 0x7f80u) == 0) sb = 0;              // below the least normal: the group is its minimum
    if (!good) sb = bb = 0x7fc0u;
    coef = sb | (bb << 16);
    codes = 0;
    if (good && sb != 0) {
        const float s = bf16_bits_to_f32(sb), b = bf16_bits_to_f32(bb), inv = 1.0f / s;
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // the correctly rounded quotient: with inv the correctly rounded
            // reciprocal, one exact remainder corrects d * inv (Markstein,
            // "Computation of elementary functions on the IBM RISC System/6000
            // processor", 1990); 3 operations for a division's 10
            const float d = x[i] - b, q0 = d * inv;
            q[i] = fmaf(fmaf(-q0, s, d), inv, q0);
        }
        // scales whose reciprocal or remainders leave the normal range
        if (s <= 0x1p-100f || s >= 0x1p100f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = (x[i] - b) / s;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = __builtin_amdgcn_fmed3f(__builtin_rintf(q[i]), 0.0f, 15.0f);
        // four codes side by side are exact in a float32
        const float q0 = fmaf(4096.0f, q[3], fmaf(256.0f, q[2], fmaf(16.0f, q[1], q[0])));
        const float q1 = fmaf(4096.0f, q[7], fmaf(256.0f, q[6], fmaf(16.0f, q[5], q[4])));
        codes = static_cast<uint32_t>(q0) | (static_cast<uint32_t>(q1) << 16);
    }
}

// A lane takes 8 channels of K and of V: both loads, and the slot's, are in
// flight together (what bounds it is how long they take).
template <typename T>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(AppendParams p)
{
    int64_t t;
    int c;
    if (!append_place(p.map, p.n, t, c)) return;     // whole runs of 8 lanes leave together
    const int64_t slot = p.slots[t];
    float x[2][8];
    load8(reinterpret_cast<const T *>(p.src[0]) + t * p.stride[0] + c, x[0]);
    load8(reinterpret_cast<const T *>(p.src[1]) + t * p.stride[1] + c, x[1]);
    const int lane = threadIdx.x & 63;
    uint32_t codes[2], coef[2];
#pragma unroll
    for (int part = 0; part < 2; ++part) quantize_group(x[part], lane, codes[part], coef[part]);
    const int64_t page = slot >> p.kv.page_shift;
    if (slot < 0 || page >= p.kv.num_pages) return;
    const int head = c >> p.kv.dim_shift, d = c & (p.kv.dim - 1);
    uint8_t *block = p.kv.data + page * p.kv.page_bytes + int64_t(head) * p.kv.block_bytes;
    const int at = static_cast<int>(slot) & ((1 << p.kv.page_shift) - 1);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        *reinterpret_cast<uint32_t *>(block + kv_part(p.kv, part) + at * (p.kv.dim / 2) + d / 2) = codes[part];
        if ((lane & 7) == 0)
            *reinterpret_cast<uint32_t *>(block + kv_coefs(p.kv, part) + at * kv_coef_bytes(p.kv.dim) + d / 16) = coef[part];
    }
}

struct ReadParams {
    char *dst[2];
    int64_t stride[2];
    const int32_t *slots;
    int64_t n;
    AppendMap map;
    KvView kv;
};

template <typename T>
__global__ __launch_bounds__(kAppendThreads) void kv_read_kernel(ReadParams p)
{
    const int part = blockIdx.y;
    if (!p.dst[part]) return;
    int64_t t;
    int c;
    if (!append_place(p.map, p.n, t, c)) return;
    const int64_t slot = p.slots[t];
    const int64_t page = slot >> p.kv.page_shift;
    const int head = c >> p.kv.dim_shift, d = c & (p.kv.dim - 1);
    float x[8];
    if (slot < 0 || page >= p.kv.num_pages) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __builtin_nanf("");
    } else {
        const uint8_t *block = p.kv.data + page * p.kv.page_bytes + int64_t(head) * p.kv.block_bytes;
        const int at = static_cast<int>(slot) & ((1 << p.kv.page_shift) - 1);
        const uint32_t codes = *reinterpret_cast<const uint32_t *>(block + kv_part(p.kv, part) + at * (p.kv.dim / 2) + d / 2);
        const uint32_t coef = *reinterpret_cast<const uint32_t *>(block + kv_coefs(p.kv, part) + at * kv_coef_bytes(p.kv.dim) +
                                                                  d / 64 * 4);
        const float s = __uint_as_float(coef << 16), b = __uint_as_float(coef & 0xffff0000u);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmaf(s, static_cast<float>((codes >> (4 * i)) & 15u), b);
    }
    store8(reinterpret_cast<T *>(p.dst[part]) + t * p.stride[part] + c, x);
}

}  // namespace qg
