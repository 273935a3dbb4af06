// Softmax cross entropy of hidden rows X [T, H] against a vocabulary W [V, H]:
// the small kernels around the products (tc_mma.cu, XENT_LOSS and XENT_GRAD).
//
//   loss       l = scale X W^T stays in TMEM: each half tile of a row leaves
//              its largest exponent and its sum of exponentials, and the
//              target's logit; `join` makes lse and the losses of them.
//   gradients  G = the gradient of l, piece by piece of the vocabulary,
//              rounded to X's type (in two parts where that is not enough);
//              dX += G W_piece and dW_piece = G^T X are plain products.  `prep` runs first, `round` last where dX was
//              summed over pieces in fp32.
//
// All of it is some microseconds beside products of 2 T H V operations each.
#include "elem.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "xent.cuh"
#include "../../include/tcgemm.h"

namespace tc {
namespace {

constexpr int JOIN_THREADS = 256;
constexpr float LN2 = 0.6931471805599453f;

// (m, s) <- the statistics of both: s 2^m + t 2^n = (..) 2^max(m, n)
__device__ __forceinline__ void merge(float &m, float &s, float n, float t)
{
    const float top = fmaxf(m, n), base = top == -INFINITY ? 0.0f : top;
    s = s * exp2_approx(m - base) + t * exp2_approx(n - base);
    m = top;
}

// Block sum in a fixed order (a tree over lanes, then one over the warps' sums);
// the result in every thread.
template <typename T>
__device__ __forceinline__ T block_sum(T v, T *buf)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) buf[warp] = v;
    __syncthreads();
    v = lane < (int)(blockDim.x >> 5) ? buf[lane] : T(0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// the sum of a block's rows and how many count, the reduced loss of them
__device__ __forceinline__ float reduced(double sum, int n, int reduction)
{
    return (float)(reduction == TC_REDUCE_MEAN && n > 0 ? sum / n : sum);
}

// A block joins `rows` neighbouring rows (a power of two up to 8: 64 bytes of
// each part), its threads the parts in turns; two floats per row and 128
// columns of the vocabulary are read once.
__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(const XentJoinArgs a, int rows)
{
    __shared__ float sm[JOIN_THREADS], ss[JOIN_THREADS];
    griddep_wait();
    griddep_launch_dependents();
    const int per = JOIN_THREADS / rows;
    const int r = threadIdx.x % rows, q = threadIdx.x / rows;
    const long long row = (long long)blockIdx.x * rows + r;
    const bool in = row < a.T;
    float m = -INFINITY, s = 0.0f;
    if (in) {
        int i = q;
        for (; i + 3 * per < a.nparts; i += 4 * per) {
            float2 p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = __ldcg(a.part + (long long)(i + j * per) * a.T + row);
#pragma unroll
            for (int j = 0; j < 4; ++j) merge(m, s, p[j].x, p[j].y);
        }
        for (; i < a.nparts; i += per) {
            const float2 p = __ldcg(a.part + (long long)i * a.T + row);
            merge(m, s, p.x, p.y);
        }
    }
    sm[threadIdx.x] = m;
    ss[threadIdx.x] = s;
    __syncthreads();
    for (int step = per / 2; step > 0; step >>= 1) {
        if (q < step) {
            merge(m, s, sm[threadIdx.x + step * rows], ss[threadIdx.x + step * rows]);
            sm[threadIdx.x] = m;
            ss[threadIdx.x] = s;
        }
        __syncthreads();
    }
    float loss = 0.0f;
    bool counted = false;
    if (q == 0 && in) {
        const float lse = (m + log2f(s)) * LN2;
        long long y;
        counted = xent_counts(a.targets, a.wide, a.vocab, row, y);
        loss = counted ? lse - a.at[row] + a.z * lse * lse : 0.0f;
        a.lse[row] = lse;
        if (a.reduction == TC_REDUCE_NONE)
            a.loss[row] = loss;
        else if (gridDim.x > 1)
            a.rows[row] = loss;
    }
    if (a.reduction != TC_REDUCE_NONE && gridDim.x == 1) {
        __shared__ double sums[JOIN_THREADS / 32];
        __shared__ int ns[JOIN_THREADS / 32];
        const double sum = block_sum((double)loss, sums);
        const int n = block_sum(counted ? 1 : 0, ns);
        if (threadIdx.x == 0) a.loss[0] = reduced(sum, n, a.reduction);
    }
}

// The reduced loss of many rows: one block, in 64 bits and a fixed order.
__global__ void __launch_bounds__(1024) total_kernel(const XentJoinArgs a)
{
    __shared__ double sums[32];
    __shared__ int ns[32];
    griddep_wait();
    griddep_launch_dependents();
    double sum = 0.0;
    int n = 0;
    for (int row = threadIdx.x; row < a.T; row += 1024) {
        long long y;
        sum += (double)a.rows[row];
        n += xent_counts(a.targets, a.wide, a.vocab, row, y) ? 1 : 0;
    }
    sum = block_sum(sum, sums);
    n = block_sum(n, ns);
    if (threadIdx.x == 0) a.loss[0] = reduced(sum, n, a.reduction);
}

constexpr int PREP_THREADS = 1024;

// Block 0 makes the rows' factors, the others copy X.
__global__ void __launch_bounds__(PREP_THREADS) prep_kernel(const XentPrepArgs a)
{
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x > 0) {
        xent_copy(a, (long long)(blockIdx.x - 1) * PREP_THREADS + threadIdx.x, (long long)(gridDim.x - 1) * PREP_THREADS);
        return;
    }
    __shared__ int ns[32];
    __shared__ float tops[32];
    float mean = 1.0f;
    if (a.reduction == TC_REDUCE_MEAN) {
        int n = 0;
        for (int t = threadIdx.x; t < a.T; t += PREP_THREADS) n += xent_counts(a, t) ? 1 : 0;
        n = block_sum(n, ns);
        mean = 1.0f / (float)max(n, 1);
    }
    float power = 1.0f;
    if (a.unscale) {
        float top = 0.0f;
        for (int t = threadIdx.x; t < a.T; t += PREP_THREADS) {
            float cp, cy;
            xent_factors(a, t, mean, cp, cy);
            top = fmaxf(top, fmaxf(fabsf(cp), fabsf(cy)));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
        __syncthreads();
        for (int w = 0; w < 32; ++w) top = fmaxf(top, tops[w]);
        power = xent_power(top);
        for (int h = threadIdx.x; h < a.H; h += PREP_THREADS) a.unscale[h] = 1.0f / power;
    }
    for (int t = threadIdx.x; t < a.T; t += PREP_THREADS) {
        float cp, cy;
        xent_factors(a, t, mean, cp, cy);
        a.cp[t] = cp * power;
        a.cy[t] = cy * power;
    }
}

__global__ void __launch_bounds__(256) round_kernel(const XentRoundArgs a)
{
    griddep_wait();
    griddep_launch_dependents();
    const long long per = (a.cols + 7) / 8, all = per * a.rows;
    const bool whole = a.cols % 8 == 0 && a.ld % 8 == 0 && (reinterpret_cast<uintptr_t>(a.dst) & 15u) == 0;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
        const long long row = i / per, col = (i - row * per) * 8, at = row * a.ld_src + col;
        float v[8];
        if (whole) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float4 x = *reinterpret_cast<const float4 *>(a.src + at + 4 * q);
                if (a.more) {
                    const float4 y = *reinterpret_cast<const float4 *>(a.more + at + 4 * q);
                    x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                }
                v[4 * q] = x.x, v[4 * q + 1] = x.y, v[4 * q + 2] = x.z, v[4 * q + 3] = x.w;
            }
            if (a.dtype == TC_F32) {
                float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(a.dst) + row * a.ld + col);
                dst[0] = make_float4(v[0], v[1], v[2], v[3]);
                dst[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.dst) + row * a.ld + col) =
                    make_uint4(pack2(v[0], v[1], a.dtype), pack2(v[2], v[3], a.dtype), pack2(v[4], v[5], a.dtype),
                               pack2(v[6], v[7], a.dtype));
            }
        } else {
            for (int j = 0; j < 8 && col + j < a.cols; ++j)
                store_c1(a.dst, row * a.ld + col + j, a.src[at + j] + (a.more ? a.more[at + j] : 0.0f), a.dtype);
        }
    }
}

unsigned blocks_for(long long items, int threads) { return (unsigned)min((items + threads - 1) / threads, 8LL * 152); }

}  // namespace

cudaError_t launch_xent_join(const XentJoinArgs &a, cudaStream_t st, int *launches)
{
    int rows = 1;
    while (rows < 8 && rows < a.T) rows *= 2;
    const unsigned grid = (unsigned)((a.T + rows - 1) / rows);
    *launches = 1;
    cudaError_t e = launch_dependent(join_kernel, dim3(grid), dim3(JOIN_THREADS), 0, st, 1u, a, rows);
    if (e != cudaSuccess || a.reduction == TC_REDUCE_NONE || grid == 1) return e;
    *launches = 2;
    return launch_dependent(total_kernel, dim3(1), dim3(1024), 0, st, 1u, a);
}

cudaError_t launch_xent_prep(const XentPrepArgs &a, cudaStream_t st)
{
    const unsigned copy = blocks_for(a.ld_clean / 8 * a.T, PREP_THREADS);
    return launch_dependent(prep_kernel, dim3(1 + copy), dim3(PREP_THREADS), 0, st, 1u, a);
}

cudaError_t launch_xent_round(const XentRoundArgs &a, cudaStream_t st)
{
    return launch_dependent(round_kernel, dim3(blocks_for((a.cols + 7) / 8 * a.rows, 256)), dim3(256), 0, st, 1u, a);
}

}  // namespace tc
