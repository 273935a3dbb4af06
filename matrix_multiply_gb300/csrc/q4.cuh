// Device helpers of the 4-bit weight kernels.
#pragma once
#include "elem.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace tc {

// Element j of a 32-bit word's eight sits at nibble (j / 2) + 4 (j % 2): a
// mask of the word shifted by 4 i leaves elements 2 i and 2 i + 1 in the low
// and high halves of a register.

// ------------------------------------------------- streaming kernels' pieces
// A piece of a 4-bit weight as the streaming kernels hold it in shared
// memory: 16 rows x Q4_SLAB k, 128 bytes a row, copied by TMA with the
// 128-byte swizzle (16-byte unit u of row r sits at u ^ (r % 8)), so that a
// warp reading one 32-bit word per lane -- word t of unit u of row g, lane =
// 4 g + t -- touches all 32 banks.  Beside the codes lie, per group, the
// scales of 24 rows and the zero points of 32 (of 16 more for two pieces
// copied at once), from the last row at or
// before the piece's first that is a multiple of 8 (16): TMA copies start at
// multiples of 16 bytes.
constexpr int Q4_SLAB = 256;
constexpr int Q4_ZERO_PITCH = Q4_ZERO_BOX;

// D(16x8, f32) = A(16x16) * B(16x8) + C, A row-major, B column-major
template <bool BF16>
__device__ __forceinline__ void q4_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                       const float (&c)[4])
{
    if constexpr (BF16) {
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
    } else {
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
    }
}

// Widened codes are code - zero for f16 and (code - zero) / 2^11 for bf16: bf16
// activations go up to fp32's largest, and a group's 128 products of up to 15
// times that must not overflow before the scale brings them down (fp16's largest
// leaves room).  Exact either way; sums of bf16 products are 2^-11 of what they
// stand for until q4_whole.
template <bool BF16>
__device__ __forceinline__ float q4_whole(float sum)
{
    return BF16 ? sum * 2048.0f : sum;
}

// What turns a row's codes into widened ones: the zero point in the biased
// form that q4_widen subtracts.
struct Q4Zero {
    uint32_t a, b;
};
template <bool BF16>
__device__ __forceinline__ Q4Zero q4_zero_form(uint32_t z)
{
    const uint32_t zz = z * 0x00010001u;
    if constexpr (BF16) return Q4Zero{0x3D803D80u | zz, 0u};             // (128 + z) / 2^11
    return Q4Zero{0x64006400u | zz, 0xD400D400u | (zz << 4)};            // 1024 + z and -(64 + z)
}

// The word's eight codes, widened, as four pairs of exact 16-bit floats
// (elements 0 1 | 2 3 | 4 5 | 6 7).  A masked nibble put under the exponent of
// 2^10 (f16) is 1024 + code, or 1024 + 16 code for the nibble above it, which
// one multiply-add brings back; bf16 has 7 fraction bits, so there every nibble
// is shifted to the bottom, under 2^-4: (128 + code) / 2^11.
template <bool BF16>
__device__ __forceinline__ void q4_widen(uint32_t w, const Q4Zero &z, uint32_t (&p)[4])
{
    if constexpr (BF16) {
        const __nv_bfloat162 zz = *reinterpret_cast<const __nv_bfloat162 *>(&z.a);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t v;
            asm("lop3.b32 %0, %1, 0x000f000f, 0x3D803D80, 0xEA;" : "=r"(v) : "r"(w >> (4 * i)));
            const __nv_bfloat162 h = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), zz);
            p[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    } else {
        const __half2 za = *reinterpret_cast<const __half2 *>(&z.a), zb = *reinterpret_cast<const __half2 *>(&z.b);
        const __half2 sixteenth = __half2half2(__ushort_as_half((unsigned short)0x2C00u));
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            uint32_t u, v;
            const uint32_t x = w >> (4 * i);
            asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xEA;" : "=r"(u) : "r"(x));
            asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xEA;" : "=r"(v) : "r"(x));
            const __half2 h0 = __hsub2(*reinterpret_cast<const __half2 *>(&u), za);
            const __half2 h1 = __hfma2(*reinterpret_cast<const __half2 *>(&v), sixteenth, zb);
            p[i] = *reinterpret_cast<const uint32_t *>(&h0);
            p[i + 1] = *reinterpret_cast<const uint32_t *>(&h1);
        }
    }
}

template <bool BF16>
__device__ __forceinline__ float q4_scale_bits(uint32_t b)
{
    return BF16 ? __uint_as_float(b << 16) : __half2float(__ushort_as_half((unsigned short)b));
}

// Where a lane (g, t) finds its share of a slab in shared memory: its word
// of unit 0 of row g (unit u: the offset ^ 16 u; row g + 8: 1024 bytes on),
// and the two rows' scales and zero points of the slab's first group
// (z0 null: none).
struct Q4Slab {
    const uint8_t *base;       // a multiple of 1024 in shared memory
    uint32_t codes;
    const uint16_t *s0, *s1;
    const uint8_t *z0, *z1;
};
__device__ __forceinline__ uint32_t q4_first_word(int g, int t) { return g * 128 + g * 16 + t * 4; }

// acc[nt] (rows g, g + 8 x X rows 8 nt + 2 t, + 1) += the slab's product with
// xf: step j's register q holds X row 8 nt + g, k = 32 j + 8 t + 2 q and + 1.
// Each group's products are summed from zero by the tensor core -- widened
// codes times 16-bit floats, exact, added in fp32 -- and join the
// accumulator times the row's scale (q4_whole is the caller's).  JOIN: the NT operands are the parts of
// one (x = part 0 + part 1), their sums join acc[0].  SP, ZP: elements between
// two groups' scales and zero points.  Every lane of the warp calls it.
template <bool BF16, bool SBF16, int NT, int G, int SP, bool JOIN = false, int ZP = Q4_ZERO_PITCH>
__device__ __forceinline__ void q4_slab(float (&acc)[JOIN ? 1 : NT][4], const Q4Slab &b, const uint32_t (&xf)[NT][8][4])
{
    constexpr int STEPS = G / 32;                  // 32-k steps per group
#pragma unroll
    for (int gr = 0; gr < Q4_SLAB / G; ++gr) {
        Q4Zero z0 = q4_zero_form<BF16>(8u), z1 = z0;
        if (b.z0) {
            z0 = q4_zero_form<BF16>((uint32_t)b.z0[gr * ZP] & 15u);
            z1 = q4_zero_form<BF16>((uint32_t)b.z1[gr * ZP] & 15u);
        }
        const float s0 = q4_scale_bits<SBF16>(b.s0[gr * SP]);
        const float s1 = q4_scale_bits<SBF16>(b.s1[gr * SP]);
        float part[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) part[nt][0] = part[nt][1] = part[nt][2] = part[nt][3] = 0.0f;
#pragma unroll
        for (int st = 0; st < STEPS; ++st) {
            const int j = gr * STEPS + st;
            const uint32_t *at = reinterpret_cast<const uint32_t *>(b.base + (b.codes ^ (uint32_t)(j << 4)));
            uint32_t p0[4], p1[4];
            q4_widen<BF16>(at[0], z0, p0);
            q4_widen<BF16>(at[256], z1, p1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint32_t lo[4] = {p0[0], p1[0], p0[1], p1[1]}, hi[4] = {p0[2], p1[2], p0[3], p1[3]};
                q4_mma<BF16>(part[nt], lo, xf[nt][j][0], xf[nt][j][1], part[nt]);
                q4_mma<BF16>(part[nt], hi, xf[nt][j][2], xf[nt][j][3], part[nt]);
            }
        }
        if constexpr (JOIN) {
#pragma unroll
            for (int nt = 1; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) part[0][e] += part[nt][e];
        }
#pragma unroll
        for (int nt = 0; nt < (JOIN ? 1 : NT); ++nt) {
            acc[nt][0] = fmaf(s0, part[nt][0], acc[nt][0]);
            acc[nt][1] = fmaf(s0, part[nt][1], acc[nt][1]);
            acc[nt][2] = fmaf(s1, part[nt][2], acc[nt][2]);
            acc[nt][3] = fmaf(s1, part[nt][3], acc[nt][3]);
        }
    }
}

// Work of one lane inside a loop that the whole warp runs: the lane whose
// `leader` is set (elect_one) arms a barrier and issues a copy.  As a
// divergent branch the same would take every address and coordinate out of
// uniform registers and back for each copy.
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }
__device__ __forceinline__ void arrive_expect_by(uint32_t bar, uint32_t bytes, uint32_t leader)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
        "r"(bytes), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void tma_load_2d_by(uint32_t dst, const void *tmap, uint32_t bar, int32_t c0, int32_t c1,
                                               uint32_t leader)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
        "\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_by(uint32_t dst, const void *tmap, uint32_t bar, int32_t c0, int32_t c1, int32_t c2,
                                               uint32_t leader)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
        "\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(leader)
        : "memory");
}

// The warps of one group (of `n` warps, several groups to a CTA) meet.
// Barrier 0 is __syncthreads'; a group of one warp needs none, so at most 8
// others are in use.
__device__ __forceinline__ void q4_group_sync(int group, int n)
{
    __syncwarp();
    if (n > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(n * 32) : "memory");
}

// Bounded waits.  A wait that runs out reports through `status` and raises
// the CTA's abort flag (where it has one), which ends the other waits of the
// CTA; the kernel then finishes without the data, its outputs undefined.
struct Q4Watch {
    volatile uint32_t *abort_flag;      // or null
    unsigned *status;
    unsigned long long timeout_ns;
};
static __device__ __noinline__ bool q4_wait_slow(uint32_t bar, uint32_t parity, const Q4Watch &w)
{
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 15u) != 0) continue;
        if (w.abort_flag && *w.abort_flag) return false;
        if (globaltimer_ns() - t0 > w.timeout_ns) {
            if (w.abort_flag) *w.abort_flag = 1u;
            *(volatile unsigned *)w.status = 0x200u;
            __threadfence_system();
            return false;
        }
    }
}
__device__ __forceinline__ bool q4_wait(uint32_t bar, uint32_t parity, const Q4Watch &w)
{
    if (mbar_try_wait(bar, parity)) return true;
    return q4_wait_slow(bar, parity, w);
}
// after an expired wait: up to 0.2 s for a copy or an MMA already under way
static __device__ __noinline__ void q4_drain(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < 200000000ull) {}
}

// 16 bytes (8 elements) of X from element k of a row, zeros past K; `vec`:
// rows are 16-byte aligned
__device__ __forceinline__ uint4 q4_load_x(const uint16_t *row, long long k, long long K, bool vec)
{
    if (vec && k + 8 <= K) return __ldg(reinterpret_cast<const uint4 *>(row + k));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (k + j < K) w[j >> 1] |= (uint32_t)row[k + j] << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A lane's share of a slab of an X row as q4_slab takes it (from element k:
// eight of every 32), zeros past K.  `whole`: 16-byte aligned rows, the slab
// inside K.  Otherwise pairs of elements (rows on 4 bytes) or single ones,
// half of them under way at a time.
// PAIRS false leaves the pairs out, where the load is part of a kernel's main loop.
template <bool PAIRS = true>
__device__ __forceinline__ void q4_load_slab(uint32_t (&xf)[8][4], const uint16_t *row, long long k, long long K, bool whole)
{
    if (whole) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(row + k) + 4 * j);
            xf[j][0] = v.x, xf[j][1] = v.y, xf[j][2] = v.z, xf[j][3] = v.w;
        }
    } else if (PAIRS && (reinterpret_cast<uintptr_t>(row) & 3u) == 0) {
        const int left = (int)min(1024LL, K - k);              // elements from the lane's first on (k is even)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = 32 * j + 2 * i;
                xf[j][i] = 0u;
                if (at + 1 < left)
                    xf[j][i] = __ldg(reinterpret_cast<const uint32_t *>(row + k + at));
                else if (at < left)
                    xf[j][i] = __ldg(row + k + at);
            }
    } else {
        const int left = (int)min(1024LL, K - k);
#pragma unroll
        for (int b = 0; b < 8; b += 4) {
            uint16_t h[4][8];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int at = 32 * (b + j) + i;
                    h[j][i] = 0;
                    if (at < left) h[j][i] = __ldg(row + k + at);
                }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) xf[b + j][i] = (uint32_t)h[j][2 * i] | (uint32_t)h[j][2 * i + 1] << 16;
        }
    }
}

}  // namespace tc
