// mx_common.hpp -- what the microscaled (MX) kernels share.
//
// An MX row is blocks of 32 consecutive elements with one scale byte s each,
// which stands for 2^(s - 127) (255: the block is NaN). Elements are e2m1 (4
// bits, two to a byte, even k in the low nibble) or e4m3 (8 bits); the formats
// are the OCP Microscaling Formats specification's, version 1.0, which the
// gfx950 matrix instructions take as operands. Rows of scales are padded to
// whole dwords.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../serve/kv_cache.hpp"

namespace qg {

constexpr int kMxBlock = 32;

// The element types, by their selector in the scaled matrix instructions.
constexpr int kMxE4M3 = 0, kMxE2M1 = 4;

template <int FMT> constexpr int kMxEmax = FMT == kMxE2M1 ? 2 : 8;          // exponent of the largest element
// Bytes of n elements.
template <int FMT> __host__ __device__ constexpr int64_t mx_bytes(int64_t n) { return FMT == kMxE2M1 ? n / 2 : n; }
__host__ __device__ constexpr int64_t mx_pitch(int64_t k) { return (k / kMxBlock + 3) / 4 * 4; }

// Division of 0 <= n < 2^31 by a number known on the host: with l = ceil(log2
// d), n * (floor(2^(31 + l) / d) + 1) >> (31 + l) is the exact quotient
// (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994).
struct FastDiv {
    uint32_t mul, shift, d;
};

inline FastDiv fast_div(uint32_t d)
{
    uint32_t l = 0;
    while ((uint64_t(1) << l) < d) ++l;
    return FastDiv{static_cast<uint32_t>((uint64_t(1) << (31 + l)) / d + 1), 31 + l, d};
}

__device__ __forceinline__ uint32_t operator/(uint32_t n, const FastDiv &f)
{
    return static_cast<uint32_t>((uint64_t(n) * f.mul) >> f.shift);
}

// v plus the value DPP brings from a lower lane (0 where there is none), and
// with it the inclusive sum over the lanes of a wave.
template <int CTRL, int ROWS>
__device__ __forceinline__ int add_lower(int v)
{
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_inclusive_sum32(int v)
{
    v = add_lower<0x111, 0xF>(v);
    v = add_lower<0x112, 0xF>(v);
    v = add_lower<0x114, 0xF>(v);
    v = add_lower<0x118, 0xF>(v);
    v = add_lower<0x142, 0xA>(v);
    return add_lower<0x143, 0xC>(v);
}

// Raw buffer resource over [base, base + bytes): a load whose offset lies
// outside the range returns zeros, so edges need no branches.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t mx_buffer(const void *base, int64_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, static_cast<int>(bytes), 0x00020000);
}
constexpr uint32_t kMxOut = 0x80000000u;   // above every range used here

constexpr int kMaxExperts = 1024;

// A wave's 64 pieces of 16 (or 4) bytes, each from its lane's offset, to LDS
// behind `dst`, one behind the other. (Plain functions: in a template the builtins
// keep the compiler's host pass from emitting the kernel.)
typedef __attribute__((address_space(3))) void *mx_lds_t;
__device__ __forceinline__ void mx_to_lds16(__amdgpu_buffer_rsrc_t buf, uint8_t *dst, uint32_t off)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (mx_lds_t)dst, 16, off, 0, 0, 0);
}
__device__ __forceinline__ void mx_to_lds4(__amdgpu_buffer_rsrc_t buf, uint8_t *dst, uint32_t off)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (mx_lds_t)dst, 4, off, 0, 0, 0);
}

// `off`, or an offset out of range when i >= n, by arithmetic only: a select
// here would be turned into a branch around the load.
__device__ __forceinline__ uint32_t mx_in_or_out(uint32_t off, int i, int n)
{
    uint32_t out = static_cast<uint32_t>(n - 1 - i) & 0x80000000u;
    asm("" : "+v"(out));
    return off | out;
}

// The wave's LDS accesses before this come before those after it.
__device__ __forceinline__ void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The value, computed where this stands: what follows from it is not kept in
// registers over the loops around.
__device__ __forceinline__ int mx_here(int v)
{
    asm volatile("" : "+v"(v));
    return v;
}

__device__ __forceinline__ int mx_here_scalar(int v)
{
    asm volatile("" : "+s"(v));
    return v;
}

}  // namespace qg
