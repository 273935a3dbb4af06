// Device helpers of the 4-bit weight kernels.
#pragma once
#include "elem.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace tc {

// Element j of a 32-bit word's eight sits at nibble (j / 2) + 4 (j % 2): a
// mask of the word shifted by 4 i leaves elements 2 i and 2 i + 1 in the low
// and high halves of a register.
__host__ __device__ constexpr int q4_nibble(int j) { return (j >> 1) + 4 * (j & 1); }

__device__ __forceinline__ float q4_scale(const Q4View &q, long long group, long long n)
{
    const uint16_t b = static_cast<const uint16_t *>(q.scales)[group * q.lds + n];
    return q.scale_bf16 ? __bfloat162float(__ushort_as_bfloat16(b)) : __half2float(__ushort_as_half(b));
}
__device__ __forceinline__ int q4_zero(const Q4View &q, long long group, long long n)
{
    return q.zeros ? (q.zeros[group * q.lds + n] & 15) : 8;
}
__device__ __forceinline__ uint32_t q4_word(const Q4View &q, long long n, long long word)
{
    return reinterpret_cast<const uint32_t *>(q.codes + n * (q.ldw >> 1))[word];
}

__device__ __forceinline__ float load_16(const void *p, long long off, int bf16)
{
    const uint16_t b = static_cast<const uint16_t *>(p)[off];
    return bf16 ? __bfloat162float(__ushort_as_bfloat16(b)) : __half2float(__ushort_as_half(b));
}

}  // namespace tc
