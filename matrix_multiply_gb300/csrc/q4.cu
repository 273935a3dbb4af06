// 4-bit weights with group scales: quantising and giving the values back.
//
// Both are bound by HBM: quantising 16-bit weights reads 2 bytes and writes
// half a byte (and the scales) per weight.  A CTA takes 16 rows x 1024 k, a
// warp a row, a lane eight consecutive k at a time -- one word of codes, one
// 16-byte load -- so codes and weights move in whole lines; a group is 4, 8
// or 16 neighbouring lanes, its extremes a few shuffles.  Scales lie n-major
// beside each other: the 16 rows' scales meet in shared memory and leave as
// 32-byte pieces.
#include "q4.cuh"

namespace tc {
namespace {

constexpr int QZ_ROWS = 16, QZ_THREADS = QZ_ROWS * 32;
constexpr int QZ_STEPS = 4, QZ_COLS = QZ_STEPS * 256;      // k of a CTA
constexpr int QZ_GROUPS = QZ_COLS / 32;                    // groups of a CTA, at most

// Eight values of a row from k, zeros past K; `vec`: 16-byte aligned rows
template <int DT>
__device__ __forceinline__ void load_w8(const void *row, long long k, long long K, bool vec, float (&v)[8])
{
    if (vec && k + 8 <= K) {
        if constexpr (DT == TC_F32) {
            const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(row) + k);
            const float4 x = __ldcs(p), y = __ldcs(p + 1);
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
        } else {
            const uint4 x = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(row) + k));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DT == TC_BF16) {
                    v[2 * i] = __uint_as_float(w[i] << 16);
                    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                } else {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                    v[2 * i] = f.x;
                    v[2 * i + 1] = f.y;
                }
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k + i < K ? load_c(row, k + i, DT) : 0.0f;
}

// round(w / s) to nearest even, as the IEEE quotient rounds.  For 16-bit w
// and s the quotient is a tie or at least 2^-17 of its size away from one, so
// w (1 / s), good to 2^-22, rounds to the same whole number unless it is a
// tie -- which the exact remainder w - r s shows -- and no division is needed.
template <bool DIVIDE>
__device__ __forceinline__ float q4_round(float w, float s, float inv, float half)
{
    if constexpr (DIVIDE) return rintf(__fdiv_rn(w, s));
    float r = rintf(w * inv);
    const float e = fmaf(-r, s, w);
    if (fabsf(e) == half) {
        const float other = r + copysignf(1.0f, e);        // the tie's other side
        r = fmodf(r, 2.0f) != 0.0f ? other : r;
    }
    return r;
}

template <int DT, bool ZEROS>
__global__ void __launch_bounds__(QZ_THREADS) q4_quantize_kernel(const Q4QuantArgs a, int lanes_log2)
{
    __shared__ uint16_t sc[QZ_GROUPS][QZ_ROWS];
    __shared__ uint8_t zp[QZ_GROUPS][QZ_ROWS];
    griddep_launch_dependents();
    griddep_wait();
    const Q4View &q = a.q;
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const long long n0 = (long long)blockIdx.x * QZ_ROWS, n = n0 + row;
    const long long k0 = (long long)blockIdx.y * QZ_COLS;
    const int es = DT == TC_F32 ? 4 : 2;
    const bool vec = (reinterpret_cast<uintptr_t>(a.W) & 15u) == 0 && (a.ld * es) % 16 == 0;
    const long long kpad = (q.K + 31) / 32 * 32;
    if (n < q.N) {
        const uint8_t *src = static_cast<const uint8_t *>(a.W) + n * a.ld * es;
        uint32_t *dst = reinterpret_cast<uint32_t *>(const_cast<uint8_t *>(q.codes) + n * (q.ldw >> 1));
        float v[QZ_STEPS][8];
#pragma unroll
        for (int i = 0; i < QZ_STEPS; ++i) load_w8<DT>(src, k0 + i * 256 + lane * 8, q.K, vec, v[i]);
#pragma unroll
        for (int i = 0; i < QZ_STEPS; ++i) {
            const long long k = k0 + i * 256 + lane * 8;
            if (k0 + i * 256 >= q.K) break;                // (the whole warp)
            // the group's extremes; a value that is not finite makes `bad` one
            float lo = 0.0f, hi = 0.0f, bad = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (ZEROS) {
                    lo = fminf(lo, v[i][j]);
                    hi = fmaxf(hi, v[i][j]);
                } else {
                    hi = fmaxf(hi, fabsf(v[i][j]));
                }
                bad = fmaf(v[i][j], 0.0f, bad);            // 0, or NaN from an infinity or a NaN on
            }
            for (int o = 1; o < (1 << lanes_log2); o <<= 1) {
                if constexpr (ZEROS) lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
                hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
                bad += __shfl_xor_sync(0xffffffffu, bad, o);
            }
            float s = ZEROS ? __fdiv_rn(hi - lo, 15.0f) : __fdiv_rn(hi, 7.0f);
            s = bad == 0.0f ? s : __int_as_float(0x7fc00000);
            uint16_t bits;
            if (q.scale_bf16) {
                bits = __bfloat16_as_ushort(__float2bfloat16_rn(s));
                s = __bfloat162float(__ushort_as_bfloat16(bits));
            } else {
                bits = __half_as_ushort(__float2half_rn(s));
                s = __half2float(__ushort_as_half(bits));
            }
            const float inv = DT == TC_F32 ? 0.0f : __fdiv_rn(1.0f, s), half = 0.5f * s;
            float z = 8.0f;
            if (ZEROS && s != 0.0f) z = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f);
            uint32_t w = 0x88888888u;                      // a scale of 0: code = zero = 8
            if (s != 0.0f) {
                w = 0u;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float c = q4_round<DT == TC_F32>(v[i][j], s, inv, half) + z;
                    w |= (uint32_t)fminf(fmaxf(c, 0.0f), 15.0f) << (4 * q4_nibble(j));
                }
            }
            if (k < kpad) dst[k / 8] = w;
            if ((lane & ((1 << lanes_log2) - 1)) == 0) {
                const int gl = (i * 32 + lane) >> lanes_log2;
                sc[gl][row] = bits;
                if constexpr (ZEROS) zp[gl][row] = (uint8_t)z;
            }
        }
    }
    __syncthreads();
    uint16_t *scales = const_cast<uint16_t *>(static_cast<const uint16_t *>(q.scales));
    uint8_t *zeros = const_cast<uint8_t *>(q.zeros);
    const long long g0 = k0 >> (3 + lanes_log2), ngroups = (q.K + q.group - 1) / q.group;
    for (int i = threadIdx.x; i < (QZ_COLS >> (3 + lanes_log2)) * QZ_ROWS; i += QZ_THREADS) {
        const int gl = i / QZ_ROWS, r = i % QZ_ROWS;
        if (g0 + gl >= ngroups || n0 + r >= q.N) continue;
        scales[(g0 + gl) * q.lds + n0 + r] = sc[gl][r];
        if constexpr (ZEROS) zeros[(g0 + gl) * q.lds + n0 + r] = zp[gl][r];
    }
}

// ---------------------------------------------------------------- dequantise

// The same shape: a word of codes per lane and step; the 16 rows of a CTA
// share the lines of the scales.
template <int DT>
__global__ void __launch_bounds__(QZ_THREADS) q4_dequantize_kernel(const Q4DequantArgs a, int group_log2)
{
    griddep_launch_dependents();
    griddep_wait();
    const Q4View &q = a.q;
    const int lane = threadIdx.x & 31;
    const long long n = (long long)blockIdx.x * QZ_ROWS + (threadIdx.x >> 5);
    const long long k0 = (long long)blockIdx.y * QZ_COLS;
    if (n >= q.N) return;
    const int es = DT == TC_F32 ? 4 : 2;
    const bool vec = (reinterpret_cast<uintptr_t>(a.V) & 15u) == 0 && (a.ld * es) % 16 == 0;
    const uint32_t *src = reinterpret_cast<const uint32_t *>(q.codes + n * (q.ldw >> 1));
    uint32_t w[QZ_STEPS];
    float s[QZ_STEPS];
    int z[QZ_STEPS];
#pragma unroll
    for (int i = 0; i < QZ_STEPS; ++i) {
        const long long k = k0 + i * 256 + lane * 8;
        w[i] = 0u, s[i] = 0.0f, z[i] = 8;
        if (k < q.K) {
            w[i] = __ldcs(src + k / 8);
            s[i] = q4_scale(q, k >> group_log2, n);
            z[i] = q4_zero(q, k >> group_log2, n);
        }
    }
#pragma unroll
    for (int i = 0; i < QZ_STEPS; ++i) {
        const long long k = k0 + i * 256 + lane * 8;
        if (k >= q.K) continue;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (float)((int)((w[i] >> (4 * q4_nibble(j))) & 15u) - z[i]) * s[i];
        const long long off = n * a.ld + k;
        if (vec && k + 8 <= q.K) {
            if constexpr (DT == TC_F32) {
                float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(a.V) + off);
                __stcs(d, make_float4(v[0], v[1], v[2], v[3]));
                __stcs(d + 1, make_float4(v[4], v[5], v[6], v[7]));
            } else {
                __stcs(reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.V) + off),
                       make_uint4(pack2(v[0], v[1], DT), pack2(v[2], v[3], DT), pack2(v[4], v[5], DT),
                                  pack2(v[6], v[7], DT)));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k + j < q.K) store_c1(a.V, off + j, v[j], DT);
        }
    }
}

// CTAs of 16 rows x 1024 k; grid.y is limited to 65535 (K below 2^26: beyond,
// a row alone would be 33 MB of codes)
bool qz_grid(const Q4View &q, dim3 *grid)
{
    const long long bx = (q.N + QZ_ROWS - 1) / QZ_ROWS, by = (q.K + QZ_COLS - 1) / QZ_COLS;
    *grid = dim3((unsigned)bx, (unsigned)by);
    return bx <= 0x7fffffffLL && by <= 65535;
}

int log2_of(int x)
{
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

template <int DT>
cudaError_t quantize(const Q4QuantArgs &a, dim3 grid, cudaStream_t st)
{
    const int lanes = log2_of(a.q.group) - 3;
    return a.q.zeros ? launch_dependent(q4_quantize_kernel<DT, true>, grid, dim3(QZ_THREADS), 0, st, 1u, a, lanes)
                     : launch_dependent(q4_quantize_kernel<DT, false>, grid, dim3(QZ_THREADS), 0, st, 1u, a, lanes);
}

}  // namespace

cudaError_t launch_q4_quantize(const Q4QuantArgs &a, cudaStream_t st)
{
    dim3 grid;
    if (!qz_grid(a.q, &grid)) return cudaErrorInvalidValue;
    switch (a.w_dtype) {
    case TC_F16: return quantize<TC_F16>(a, grid, st);
    case TC_BF16: return quantize<TC_BF16>(a, grid, st);
    default: return quantize<TC_F32>(a, grid, st);
    }
}

cudaError_t launch_q4_dequantize(const Q4DequantArgs &a, cudaStream_t st)
{
    dim3 grid;
    if (!qz_grid(a.q, &grid)) return cudaErrorInvalidValue;
    const int g = log2_of(a.q.group);
    switch (a.v_dtype) {
    case TC_F16: return launch_dependent(q4_dequantize_kernel<TC_F16>, grid, dim3(QZ_THREADS), 0, st, 1u, a, g);
    case TC_BF16: return launch_dependent(q4_dequantize_kernel<TC_BF16>, grid, dim3(QZ_THREADS), 0, st, 1u, a, g);
    default: return launch_dependent(q4_dequantize_kernel<TC_F32>, grid, dim3(QZ_THREADS), 0, st, 1u, a, g);
    }
}

}  // namespace tc
