// A mixture-of-experts layer for a few tokens over 4-bit weights: router,
// choice of experts, gated products, down products and their weighted sum.
#include "q4.cuh"

namespace tc {
namespace {

constexpr int MOE_THREADS = 256;
constexpr int MOE_WARPS = MOE_THREADS / 32;

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// logits[t, e], one warp each
__global__ void __launch_bounds__(MOE_THREADS) moe_router_kernel(const MoeArgs a)
{
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int i = blockIdx.x * MOE_WARPS + (threadIdx.x >> 5);
    if (i >= a.T * a.E) return;
    const int t = i / a.E, e = i - t * a.E;
    float s = 0.0f;
    for (int h = lane; h < a.H; h += 32)
        s = fmaf(load_16(a.X, t * a.ldx + h, a.x_bf16), load_c(a.R, e * a.ldr + h, a.r_dtype), s);
    s = warp_sum(s);
    if (lane == 0) a.logits[i] = s;
}

// One warp per token: top_k rounds of an argmax over the logits (a NaN
// counts as the largest, ties go to the lowest index), then their softmax.
__global__ void __launch_bounds__(32) moe_topk_kernel(const MoeArgs a)
{
    griddep_launch_dependents();
    griddep_wait();
    constexpr int PER = TC_MOE_MAX_EXPERTS / 32;
    const int lane = threadIdx.x, t = blockIdx.x;
    float l[PER];
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int e = q * 32 + lane;
        l[q] = e < a.E ? a.logits[t * a.E + e] : -INFINITY;
        top = fmaxf(top, l[q]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    unsigned taken = 0;      // bit q: this lane's value q is chosen
#pragma unroll
    for (int q = 0; q < PER; ++q)
        if (q * 32 + lane < a.E) sum += expf(l[q] - top);
    sum = warp_sum(sum);
    float chosen = 0.0f, mine = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        float bv = -INFINITY;
        int be = 0x7fffffff;
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int e = q * 32 + lane;
            if (e >= a.E || (taken >> q & 1u)) continue;
            const float v = isnan(l[q]) ? INFINITY : l[q];
            if (be == 0x7fffffff || v > bv) bv = v, be = e;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
            const int oe = __shfl_xor_sync(0xffffffffu, be, o);
            if (oe != 0x7fffffff && (be == 0x7fffffff || ov > bv || (ov == bv && oe < be))) bv = ov, be = oe;
        }
        if ((be & 31) == lane) taken |= 1u << (be >> 5);
        const float e = expf(a.logits[t * a.E + be] - top);
        chosen += e;
        if (lane == j) mine = e;
        if (lane == 0) a.ids[t * a.k + j] = be;
    }
    if (lane < a.k) a.p[t * a.k + lane] = mine / (a.renorm ? chosen : sum);
}

// sum over k of W[n, k] x[k], x given by a function; the whole warp
template <typename X>
__device__ __forceinline__ float row_dot(const Q4View &q, long long n, int lane, X x)
{
    float acc = 0.0f;
    const long long words = (q.K + 7) / 8;
    for (long long wi = lane; wi < words; wi += 32) {
        const uint32_t w = q4_word(q, n, wi);
        const long long k = wi * 8;
        const int z = q4_zero(q, k / q.group, n);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (k + j < q.K) sum = fmaf((float)((int)((w >> (4 * q4_nibble(j))) & 15u) - z), x(k + j), sum);
        acc = fmaf(q4_scale(q, k / q.group, n), sum, acc);
    }
    return warp_sum(acc);
}

// h[t, j, i], one warp each
__global__ void __launch_bounds__(MOE_THREADS) moe_gate_up_kernel(const MoeArgs a)
{
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * MOE_WARPS + (threadIdx.x >> 5);
    if (w >= (long long)a.T * a.k * a.I) return;
    const int pair = (int)(w / a.I), i = (int)(w - (long long)pair * a.I);
    const long long row = (long long)a.ids[pair] * 2 * a.I + i;
    const long long x0 = (pair / a.k) * a.ldx;
    auto x = [&](long long k) { return load_16(a.X, x0 + k, a.x_bf16); };
    const float g = row_dot(a.w1, row, lane, x), u = row_dot(a.w1, row + a.I, lane, x);
    if (lane == 0) a.h[w] = g / (1.0f + expf(-g)) * u;
}

// Y[t, n], one warp each
__global__ void __launch_bounds__(MOE_THREADS) moe_down_kernel(const MoeArgs a)
{
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * MOE_WARPS + (threadIdx.x >> 5);
    if (w >= (long long)a.T * a.H) return;
    const int t = (int)(w / a.H), n = (int)(w - (long long)t * a.H);
    float y = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        const int pair = t * a.k + j;
        const float *h = a.h + (long long)pair * a.I;
        y = fmaf(a.p[pair], row_dot(a.w2, (long long)a.ids[pair] * a.H + n, lane, [&](long long k) { return h[k]; }), y);
    }
    if (lane == 0) store_c1(a.Y, t * a.ldy + n, y, a.y_dtype);
}

}  // namespace

int moe_launches() { return 4; }

cudaError_t launch_moe(const MoeArgs &a, cudaStream_t st)
{
    auto blocks = [](long long warps) { return dim3((unsigned)((warps + MOE_WARPS - 1) / MOE_WARPS)); };
    if ((long long)a.T * a.k * a.I / MOE_WARPS > 0x7ffffff0LL) return cudaErrorInvalidValue;
    cudaError_t e;
    if ((e = launch_dependent(moe_router_kernel, blocks(a.T * a.E), dim3(MOE_THREADS), 0, st, 1u, a)) != cudaSuccess)
        return e;
    if ((e = launch_dependent(moe_topk_kernel, dim3((unsigned)a.T), dim3(32), 0, st, 1u, a)) != cudaSuccess) return e;
    if ((e = launch_dependent(moe_gate_up_kernel, blocks((long long)a.T * a.k * a.I), dim3(MOE_THREADS), 0, st, 1u,
                              a)) != cudaSuccess)
        return e;
    return launch_dependent(moe_down_kernel, blocks((long long)a.T * a.H), dim3(MOE_THREADS), 0, st, 1u, a);
}

}  // namespace tc
