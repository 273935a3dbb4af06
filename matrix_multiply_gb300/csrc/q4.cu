// 4-bit weights with group scales: quantising and giving the values back.
#include "q4.cuh"

namespace tc {
namespace {

constexpr int Q4_THREADS = 256;

// ------------------------------------------------------------------ quantise

// Rounding to nearest even throughout; the quotient is the IEEE one, so that
// the code of a 16-bit weight is that of the exact quotient.
__device__ __forceinline__ uint32_t q4_code(float w, float s, float z)
{
    if (s == 0.0f) return 8u;
    const float c = rintf(__fdiv_rn(w, s)) + z;
    return (uint32_t)fminf(fmaxf(c, 0.0f), 15.0f);
}

__global__ void __launch_bounds__(Q4_THREADS) q4_quantize_kernel(const Q4QuantArgs a)
{
    griddep_launch_dependents();
    griddep_wait();
    const Q4View &q = a.q;
    const long long ngroups = (q.K + q.group - 1) / q.group;
    const long long i = (long long)blockIdx.x * Q4_THREADS + threadIdx.x;
    if (i >= ngroups * q.N) return;
    const long long n = i / ngroups, gi = i - n * ngroups;
    const long long k0 = gi * q.group, k1 = min(q.K, k0 + q.group);
    const long long kpad = min((q.K + 31) / 32 * 32, k0 + q.group);
    float lo = 0.0f, hi = 0.0f;
    bool finite = true;
    for (long long k = k0; k < k1; ++k) {
        const float w = load_c(a.W, n * a.ld + k, a.w_dtype);
        lo = fminf(lo, w);
        hi = fmaxf(hi, w);
        finite = finite && isfinite(w);
    }
    float s = q.zeros ? __fdiv_rn(hi - lo, 15.0f) : __fdiv_rn(fmaxf(hi, -lo), 7.0f);
    if (!finite) s = __int_as_float(0x7fc00000);
    uint16_t bits;
    if (q.scale_bf16) {
        bits = __bfloat16_as_ushort(__float2bfloat16_rn(s));
        s = __bfloat162float(__ushort_as_bfloat16(bits));
    } else {
        bits = __half_as_ushort(__float2half_rn(s));
        s = __half2float(__ushort_as_half(bits));
    }
    float z = 8.0f;
    if (q.zeros && s != 0.0f) z = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f);
    const_cast<uint16_t *>(static_cast<const uint16_t *>(q.scales))[gi * q.lds + n] = bits;
    if (q.zeros) const_cast<uint8_t *>(q.zeros)[gi * q.lds + n] = (uint8_t)z;
    uint32_t *row = reinterpret_cast<uint32_t *>(const_cast<uint8_t *>(q.codes) + n * (q.ldw >> 1));
    for (long long k = k0; k < kpad; k += 8) {
        uint32_t w = 0;
        for (int j = 0; j < 8; ++j) {
            const float v = k + j < k1 ? load_c(a.W, n * a.ld + k + j, a.w_dtype) : 0.0f;
            w |= q4_code(v, s, z) << (4 * q4_nibble(j));
        }
        row[k / 8] = w;
    }
}

// ---------------------------------------------------------------- dequantise

__global__ void __launch_bounds__(Q4_THREADS) q4_dequantize_kernel(const Q4DequantArgs a)
{
    griddep_launch_dependents();
    griddep_wait();
    const Q4View &q = a.q;
    const long long words = (q.K + 7) / 8;
    const long long i = (long long)blockIdx.x * Q4_THREADS + threadIdx.x;
    if (i >= words * q.N) return;
    const long long n = i / words, wi = i - n * words, k = wi * 8;
    const uint32_t w = q4_word(q, n, wi);
    const float s = q4_scale(q, k / q.group, n);
    const int z = q4_zero(q, k / q.group, n);
    for (int j = 0; j < 8; ++j)
        if (k + j < q.K)
            store_c1(a.V, n * a.ld + k + j, (float)((int)((w >> (4 * q4_nibble(j))) & 15u) - z) * s, a.v_dtype);
}

}  // namespace

cudaError_t launch_q4_quantize(const Q4QuantArgs &a, cudaStream_t st)
{
    const long long n = (a.q.K + a.q.group - 1) / a.q.group * a.q.N, blocks = (n + Q4_THREADS - 1) / Q4_THREADS;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_dependent(q4_quantize_kernel, dim3((unsigned)blocks), dim3(Q4_THREADS), 0, st, 1u, a);
}

cudaError_t launch_q4_dequantize(const Q4DequantArgs &a, cudaStream_t st)
{
    const long long n = (a.q.K + 7) / 8 * a.q.N, blocks = (n + Q4_THREADS - 1) / Q4_THREADS;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_dependent(q4_dequantize_kernel, dim3((unsigned)blocks), dim3(Q4_THREADS), 0, st, 1u, a);
}

}  // namespace tc
