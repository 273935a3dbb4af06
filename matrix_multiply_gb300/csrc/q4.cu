// 4-bit weights with group scales: quantising and giving the values back.
//
// Quantising 16-bit weights reads 2 bytes and writes half a byte (and the
// scales) per weight, and back.  A CTA takes 16 rows, a warp a row, a lane
// eight consecutive k at a time -- one word of codes, one 16-byte load -- so
// codes and weights move in whole lines; a group is 4, 8 or 16 neighbouring
// lanes, its extremes a few shuffles, its scale worked out by one of them.
// Scales lie n-major beside each other: the 16 rows' scales meet in shared
// memory and leave as 32-byte pieces.
//
// What bounds it: reading back, HBM; quantising, issue -- 154 instructions for
// a warp's 256 weights, 24 of them the test for exact ties of the rounding.
// Measured, quantising and reading back together: 65536 x 4096 f16, groups of
// 64 with zero points, 288 us for 1.37 GB, 71% of a plain copy's rate (162 and
// 139 us, 4.1 and 4.9 TB/s, under the profiler); 4096 x 4096 bf16 24 us;
// 1001 x 2999 fp32 with padded rows 15 us.
#include "q4.cuh"

namespace tc {
namespace {

constexpr int QZ_ROWS = 16, QZ_THREADS = QZ_ROWS * 32;
constexpr int QZ_STEPS = 4, QZ_COLS = QZ_STEPS * 256;      // k of a CTA (dequantising)
// k steps of a warp when quantising: as many as its registers hold (four for
// 16-bit weights: 65536 x 4096 both ways 348 us for 288)
template <int DT>
constexpr int QZ_N = DT == TC_F32 ? 4 : 8;

// What a lane holds of a step of its warp's row -- 256 k, lane l the eight
// from 8 l -- as stored: four words of 16-bit pairs, or eight of fp32.
template <int DT>
constexpr int QZ_RAW = DT == TC_F32 ? 8 : 4;

// Rows off 16 bytes (or the last piece of one) are read element by element,
// neighbouring lanes neighbouring elements, zeros past K, and change places
// through shared memory (`buf`, 8 x 33 words of the warp's own: element 8 l +
// j at 33 j + l).
template <int DT>
__device__ __forceinline__ void load_step(const void *row, long long k0, long long K, bool vec, uint32_t *buf,
                                          uint32_t (&raw)[QZ_RAW<DT>])
{
    const int lane = threadIdx.x & 31;
    if (vec && k0 + 256 <= K) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(row) + k0 * (DT == TC_F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < QZ_RAW<DT> / 4; ++i) {
            const uint4 x = __ldcs(p + lane * (QZ_RAW<DT> / 4) + i);
            raw[4 * i] = x.x, raw[4 * i + 1] = x.y, raw[4 * i + 2] = x.z, raw[4 * i + 3] = x.w;
        }
        return;
    }
    uint32_t x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const long long k = k0 + i * 32 + lane;
        x[i] = 0u;
        if (k < K) x[i] = DT == TC_F32 ? static_cast<const uint32_t *>(row)[k] : (uint32_t)static_cast<const uint16_t *>(row)[k];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = i * 32 + lane;
        buf[33 * (e & 7) + (e >> 3)] = x[i];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = buf[33 * i + lane];
        if constexpr (DT == TC_F32)
            raw[i] = b;
        else
            raw[i >> 1] = i & 1 ? raw[i >> 1] | b << 16 : b;
    }
}

template <int DT>
__device__ __forceinline__ void to_floats(const uint32_t (&raw)[QZ_RAW<DT>], float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < QZ_RAW<DT>; ++i) {
        if constexpr (DT == TC_F32) {
            v[i] = __uint_as_float(raw[i]);
        } else if constexpr (DT == TC_BF16) {
            v[2 * i] = __uint_as_float(raw[i] << 16);
            v[2 * i + 1] = __uint_as_float(raw[i] & 0xffff0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&raw[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

// max(-w, 0) and max(w, 0) over a group, or, both, max |w|; a NaN wins.  The
// group is 1 << LOG2 neighbouring lanes.  16-bit weights are compared as
// pairs, and both extremes travel in one register.
struct QzExtremes {
    float neg, pos;
};
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
template <int DT>
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b)
{
    uint32_t r;
    if constexpr (DT == TC_BF16)
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <int DT, bool ZEROS, int LOG2>
__device__ __forceinline__ void extremes(const uint32_t (&raw)[QZ_RAW<DT>], uint32_t (&out)[DT == TC_F32 && ZEROS ? 2 : 1])
{
    if constexpr (DT == TC_F32) {
        float neg = 0.0f, pos = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = __uint_as_float(raw[i]);
            pos = max_nan(pos, ZEROS ? v : fabsf(v));
            if constexpr (ZEROS) neg = max_nan(neg, -v);
        }
#pragma unroll
        for (int o = 1; o < 1 << LOG2; o <<= 1) {
            pos = max_nan(pos, __shfl_xor_sync(0xffffffffu, pos, o));
            if constexpr (ZEROS) neg = max_nan(neg, __shfl_xor_sync(0xffffffffu, neg, o));
        }
        out[0] = __float_as_uint(pos);
        if constexpr (ZEROS) out[1] = __float_as_uint(neg);
    } else {
        constexpr uint32_t SIGN = 0x80008000u;
        uint32_t m = 0u;
        if constexpr (ZEROS) {
            uint32_t pos = 0u, neg = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                pos = max2_nan<DT>(pos, raw[i]);
                neg = max2_nan<DT>(neg, raw[i] ^ SIGN);
            }
            // low half: -w, high half: w
            m = max2_nan<DT>(__byte_perm(neg, pos, 0x5410u), __byte_perm(neg, pos, 0x7632u));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) m = max2_nan<DT>(m, raw[i] & ~SIGN);
            m = max2_nan<DT>(m, __byte_perm(m, 0u, 0x1032u));
        }
#pragma unroll
        for (int o = 1; o < 1 << LOG2; o <<= 1) m = max2_nan<DT>(m, __shfl_xor_sync(0xffffffffu, m, o));
        out[0] = m;
    }
}
template <int DT, bool ZEROS>
__device__ __forceinline__ QzExtremes to_extremes(const uint32_t (&x)[DT == TC_F32 && ZEROS ? 2 : 1])
{
    if constexpr (DT == TC_F32) {
        return QzExtremes{__uint_as_float(x[ZEROS ? 1 : 0]), __uint_as_float(x[0])};
    } else if constexpr (DT == TC_BF16) {
        return QzExtremes{__uint_as_float(x[0] << 16), __uint_as_float(x[0] & 0xffff0000u)};
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x[0]));
        return QzExtremes{f.x, f.y};
    }
}

// Whole numbers are rounded by adding 1.5 2^23: the sum's low bits are the
// number, to nearest even.
constexpr float QZ_MAGIC = 12582912.0f;

// The codes round(w / s) + z, clamped to 0 .. 15, of the eight values, as a
// word.  DIVIDE: by the IEEE quotient.  Otherwise -- 16-bit weights, whose
// quotient by a 16-bit scale is a tie or at least 2^-17 of its size away from
// one -- w (1 / s), good to 2^-22, rounds to the same number unless it is a
// tie, which the exact remainder w - r s = s / 2 shows; then the quotient is
// taken after all.
template <bool DIVIDE>
__device__ __forceinline__ uint32_t q4_word_of(const float (&v)[8], float s, float inv, int z)
{
    float m[8];
    bool tie = isinf(inv);                                 // (a bf16 scale below 2^-128)
    const float half = 0.5f * s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (DIVIDE) {
            m[i] = fminf(fmaxf(__fdiv_rn(v[i], s), -16.0f), 16.0f) + QZ_MAGIC;
        } else {
            m[i] = fmaf(v[i], inv, QZ_MAGIC);
            const float e = fmaf(-(m[i] - QZ_MAGIC), s, v[i]);
            tie |= fabsf(e) == half;
        }
    }
    if (!DIVIDE && tie) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = rintf(__fdiv_rn(v[i], s)) + QZ_MAGIC;
    }
    // pairs of elements in halves of a register: + z, then clamped, two at a time
    const uint32_t zz = (uint32_t)z * 0x00010001u;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t p = __byte_perm(__float_as_uint(m[2 * i]), __float_as_uint(m[2 * i + 1]), 0x5410u);
        w |= __viaddmin_s16x2_relu(p, zz, 0x000f000fu) << (4 * i);
    }
    return w;
}

template <int DT, bool ZEROS, int LOG2>
__global__ void __launch_bounds__(QZ_THREADS, 2) q4_quantize_kernel(const Q4QuantArgs a)
{
    constexpr int STEPS = QZ_N<DT>, COLS = STEPS * 256;
    constexpr int PER = 32 >> LOG2;                            // groups of a warp's step
    constexpr int GROUPS = STEPS * PER;                     // and of its row
    constexpr int TURNS = (GROUPS + 31) / 32;                  // of a lane for each group
    __shared__ uint16_t sc[GROUPS][QZ_ROWS];
    __shared__ uint8_t zp[GROUPS][QZ_ROWS];
    __shared__ uint32_t bufs[QZ_ROWS][8 * 33];
    griddep_launch_dependents();
    griddep_wait();
    const Q4View &q = a.q;
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const long long n0 = (long long)blockIdx.x * QZ_ROWS, n = n0 + row;
    const long long k0 = (long long)blockIdx.y * COLS;
    const int es = DT == TC_F32 ? 4 : 2;
    const bool vec = (reinterpret_cast<uintptr_t>(a.W) & 15u) == 0 && (a.ld * es) % 16 == 0;
    if (n < q.N) {
        const uint8_t *src = static_cast<const uint8_t *>(a.W) + n * a.ld * es;
        const int steps = (int)min((long long)STEPS, (q.K - k0 + 255) / 256);
        uint32_t raw[STEPS][QZ_RAW<DT>];
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
#pragma unroll
            for (int j = 0; j < QZ_RAW<DT>; ++j) raw[i][j] = 0u;
            if (i < steps) load_step<DT>(src, k0 + i * 256, q.K, vec, bufs[row], raw[i]);
        }
        // lane l takes the groups l, l + 32, ... of the row: their scales,
        // computed once, and handed back to the groups' lanes
        uint32_t ext[TURNS][DT == TC_F32 && ZEROS ? 2 : 1] = {};
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            uint32_t x[DT == TC_F32 && ZEROS ? 2 : 1];
            extremes<DT, ZEROS, LOG2>(raw[i], x);
#pragma unroll
            for (int j = 0; j < (DT == TC_F32 && ZEROS ? 2 : 1); ++j) {
                const uint32_t y = __shfl_sync(0xffffffffu, x[j], (lane & (PER - 1)) << LOG2);
                if (lane / PER == i % (32 / PER)) ext[i * PER / 32][j] = y;
            }
        }
        float div[TURNS], inv[TURNS];
        int z[TURNS];
#pragma unroll
        for (int t = 0; t < TURNS; ++t) {
            const QzExtremes e = to_extremes<DT, ZEROS>(ext[t]);
            float s = ZEROS ? __fdiv_rn(e.pos + e.neg, 15.0f) : __fdiv_rn(e.pos, 7.0f);
            if (!(e.pos < INFINITY && e.neg < INFINITY)) s = __int_as_float(0x7fc00000);
            uint16_t bits;
            if (q.scale_bf16) {
                bits = __bfloat16_as_ushort(__float2bfloat16_rn(s));
                s = __bfloat162float(__ushort_as_bfloat16(bits));
            } else {
                bits = __half_as_ushort(__float2half_rn(s));
                s = __half2float(__ushort_as_half(bits));
            }
            // a scale of 0 is used as infinity: every quotient is then 0, the
            // code the zero point 8
            div[t] = s != 0.0f ? s : __int_as_float(0x7f800000);
            inv[t] = DT == TC_F32 ? 0.0f : __fdiv_rn(1.0f, div[t]);
            z[t] = 8;
            if (ZEROS && s != 0.0f) z[t] = (int)fminf(fmaxf(rintf(__fdiv_rn(e.neg, s)), 0.0f), 15.0f);
            if (t * 32 + lane < GROUPS) {
                sc[t * 32 + lane][row] = bits;
                if constexpr (ZEROS) zp[t * 32 + lane][row] = (uint8_t)z[t];
            }
        }
        uint32_t *dst = reinterpret_cast<uint32_t *>(const_cast<uint8_t *>(q.codes) + n * (q.ldw >> 1)) + k0 / 8 + lane;
        const int words = (int)min((long long)COLS / 8, ((q.K + 31) / 32 * 32 - k0) / 8) - lane;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            if (i >= steps) break;                             // (the whole warp)
            const int turn = i * PER / 32, from = (i * PER + (lane >> LOG2)) % 32;
            float v[8];
            to_floats<DT>(raw[i], v);
            const uint32_t w = q4_word_of<DT == TC_F32>(v, __shfl_sync(0xffffffffu, div[turn], from), __shfl_sync(0xffffffffu, inv[turn], from),
                                                        ZEROS ? __shfl_sync(0xffffffffu, z[turn], from) : 8);
            if (32 * i < words) dst[32 * i] = w;
        }
    }
    __syncthreads();
    uint16_t *scales = const_cast<uint16_t *>(static_cast<const uint16_t *>(q.scales));
    uint8_t *zeros = const_cast<uint8_t *>(q.zeros);
    const long long g0 = k0 >> (3 + LOG2), ngroups = (q.K + q.group - 1) / q.group;
    for (int i = threadIdx.x; i < GROUPS * QZ_ROWS; i += QZ_THREADS) {
        const int gl = i / QZ_ROWS, r = i % QZ_ROWS;
        if (g0 + gl >= ngroups || n0 + r >= q.N) continue;
        scales[(g0 + gl) * q.lds + n0 + r] = sc[gl][r];
        if constexpr (ZEROS) zeros[(g0 + gl) * q.lds + n0 + r] = zp[gl][r];
    }
}

// ---------------------------------------------------------------- dequantise

// The same shape: a word of codes per lane and step; the 16 rows of a CTA
// share the lines of the scales.  The whole numbers code - zero come as
// exact f16 pairs (q4_widen), times the scale in fp32.
template <int DT>
__global__ void __launch_bounds__(QZ_THREADS, 4) q4_dequantize_kernel(const Q4DequantArgs a, int group_log2)
{
    __shared__ float bufs[QZ_ROWS][8 * 33];
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
    const uint16_t *scales = static_cast<const uint16_t *>(q.scales) + n;
    uint32_t w[QZ_STEPS];
    uint16_t s[QZ_STEPS];
    uint8_t z[QZ_STEPS];
#pragma unroll
    for (int i = 0; i < QZ_STEPS; ++i) {
        const long long k = k0 + i * 256 + lane * 8;
        w[i] = 0u, s[i] = 0, z[i] = 8;
        if (k < q.K) {
            w[i] = __ldcs(src + k / 8);
            s[i] = scales[(k >> group_log2) * q.lds];
            if (q.zeros) z[i] = q.zeros[(k >> group_log2) * q.lds + n];
        }
    }
#pragma unroll
    for (int i = 0; i < QZ_STEPS; ++i) {
        const long long ks = k0 + i * 256, k = ks + lane * 8;
        if (ks >= q.K) break;                                  // (the whole warp)
        uint32_t p[4];
        q4_widen<false>(w[i], q4_zero_form<false>(z[i] & 15u), p);
        const float f = q.scale_bf16 ? q4_scale_bits<true>(s[i]) : q4_scale_bits<false>(s[i]);
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&p[j]));
            v[2 * j] = x.x * f;
            v[2 * j + 1] = x.y * f;
        }
        const long long off = n * a.ld + k;
        if (vec && ks + 256 <= q.K) {
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
            // neighbouring lanes store neighbouring elements (see load_step)
            float *buf = bufs[threadIdx.x >> 5];
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) buf[33 * j + lane] = v[j];
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = j * 32 + lane;
                if (ks + e < q.K) store_c1(a.V, n * a.ld + ks + e, buf[33 * (e & 7) + (e >> 3)], DT);
            }
        }
    }
}

// CTAs of 16 rows x `cols` k; grid.y is limited to 65535, which
// Q4_MATRIX_MAX_K keeps to
bool qz_grid(const Q4View &q, int cols, dim3 *grid)
{
    const long long bx = (q.N + QZ_ROWS - 1) / QZ_ROWS, by = (q.K + cols - 1) / cols;
    *grid = dim3((unsigned)bx, (unsigned)by);
    return bx <= 0x7fffffffLL && by <= 65535;
}

int log2_of(int x)
{
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

template <int DT, bool ZEROS>
cudaError_t quantize_group(const Q4QuantArgs &a, dim3 grid, cudaStream_t st)
{
    switch (a.q.group) {
    case 32: return launch_dependent(q4_quantize_kernel<DT, ZEROS, 2>, grid, dim3(QZ_THREADS), 0, st, 1u, a);
    case 64: return launch_dependent(q4_quantize_kernel<DT, ZEROS, 3>, grid, dim3(QZ_THREADS), 0, st, 1u, a);
    default: return launch_dependent(q4_quantize_kernel<DT, ZEROS, 4>, grid, dim3(QZ_THREADS), 0, st, 1u, a);
    }
}

template <int DT>
cudaError_t quantize(const Q4QuantArgs &a, dim3 grid, cudaStream_t st)
{
    return a.q.zeros ? quantize_group<DT, true>(a, grid, st) : quantize_group<DT, false>(a, grid, st);
}

}  // namespace

cudaError_t launch_q4_quantize(const Q4QuantArgs &a, cudaStream_t st)
{
    dim3 grid;
    if (!qz_grid(a.q, a.w_dtype == TC_F32 ? QZ_N<TC_F32> * 256 : QZ_N<TC_BF16> * 256, &grid)) return cudaErrorInvalidValue;
    switch (a.w_dtype) {
    case TC_F16: return quantize<TC_F16>(a, grid, st);
    case TC_BF16: return quantize<TC_BF16>(a, grid, st);
    default: return quantize<TC_F32>(a, grid, st);
    }
}

cudaError_t launch_q4_dequantize(const Q4DequantArgs &a, cudaStream_t st)
{
    dim3 grid;
    if (!qz_grid(a.q, QZ_COLS, &grid)) return cudaErrorInvalidValue;
    const int g = log2_of(a.q.group);
    switch (a.v_dtype) {
    case TC_F16: return launch_dependent(q4_dequantize_kernel<TC_F16>, grid, dim3(QZ_THREADS), 0, st, 1u, a, g);
    case TC_BF16: return launch_dependent(q4_dequantize_kernel<TC_BF16>, grid, dim3(QZ_THREADS), 0, st, 1u, a, g);
    default: return launch_dependent(q4_dequantize_kernel<TC_F32>, grid, dim3(QZ_THREADS), 0, st, 1u, a, g);
    }
}

}  // namespace tc
