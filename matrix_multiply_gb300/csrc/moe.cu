// A mixture-of-experts layer for a few tokens over 4-bit weights, in one
// cooperative launch of one CTA per SM.  It is bound by the stream of the
// chosen experts' codes and, for one or two tokens, by its three dependent
// stages, so the stages are parts of one kernel:
//   0  router: logits[t, e] in fp32, an expert per CTA; grid barrier
//   1  every CTA chooses the experts of all tokens for itself, lists the
//      tokens of each chosen expert in entries of at most 8, and takes an
//      equal share of the (entry, 8 rows of inter) units: 8 gate and 8 up rows
//      as the 16 rows of one mma.sync operand, the entry's tokens as its 8
//      columns, so a lane's gate and up sums meet in silu(gate) * up; grid
//      barrier
//   2  every CTA owns rows of hidden: the down products of all entries, added
//      with the tokens' weights in shared memory, per warp in a fixed order
// The codes go through a TMA ring per warp; its copies run ahead across the
// second barrier, since which weights stage 2 reads does not depend on h.  h
// is kept as two bf16 parts, h = hi + lo (16 bits of significand, any
// exponent), multiplied one after the other.  Deterministic: lists in index
// order, sums in fixed orders.
#include "q4.cuh"

#include <atomic>

namespace tc {
namespace {

constexpr int MO_WARPS = 16, MO_THREADS = MO_WARPS * 32;
constexpr int MO_STAGES = 3;
constexpr int MO_SCALE_AT = 2048, MO_ZERO_AT = 2560;     // codes 2 x 8 rows; scales, zero points 2 x 256 bytes
constexpr int MO_STAGE_BYTES = 3072;
constexpr int MO_RING = MO_WARPS * MO_STAGES * MO_STAGE_BYTES;
constexpr int MO_TILE_LD = 20, MO_TILE = 8 * MO_TILE_LD; // floats: a unit's partial tile, 8 tokens x 16 rows
constexpr int MO_HOLD = 6;                               // units whose partial tiles are held before they are added
constexpr int MO_PANEL = 32;                             // rows of hidden per stage-2 panel
constexpr int MO_PAIRS = TC_MOE_MAX_TOKENS * TC_MOE_MAX_TOPK;
constexpr int MO_SUMS = MO_WARPS * TC_MOE_MAX_TOKENS * MO_PANEL * 4;
static_assert(MO_HOLD * MO_WARPS * MO_TILE * 4 <= MO_SUMS, "stage 1's tiles share stage 2's space");
static_assert(MO_PAIRS <= MO_THREADS && TC_MOE_MAX_EXPERTS <= MO_THREADS && TC_MOE_MAX_TOKENS <= 32, "one thread each");

struct MoeLists {
    uint32_t mask[TC_MOE_MAX_EXPERTS];       // tokens that chose the expert
    uint16_t off[TC_MOE_MAX_EXPERTS];        // the expert's first place in `pair`
    uint16_t pair[MO_PAIRS];                 // t * top_k + j, by expert, then token
    uint16_t id[MO_PAIRS];                   // of pair t * top_k + j: the expert
    float p[MO_PAIRS];                       //   and its weight
    uint16_t ent_e[MO_PAIRS], ent_at[MO_PAIRS];   // entries: expert, first place in `pair`
    uint8_t ent_n[MO_PAIRS];                      //   and number of tokens (1 .. 8)
    uint32_t scan[MO_WARPS];
    int entries;
    float red[MO_WARPS][8];
};
constexpr int MO_SMEM = 1024 + MO_RING + MO_SUMS + (int)sizeof(MoeLists) + MO_WARPS * MO_STAGES * 8 + 16;
static_assert(MO_SMEM <= SMEM_LIMIT, "one CTA per SM");

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// All CTAs of the grid (a cooperative launch: all are resident).  sync[0]
// counts arrivals, the last of which resets it and moves sync[1] on.  The wait
// is bounded: past the limit the kernel reports and goes on, its outputs
// undefined.
__device__ __forceinline__ void grid_arrive(unsigned *sync, unsigned &gen)
{
    __syncthreads();
    if (threadIdx.x == 0) {
        gen = *(volatile unsigned *)(sync + 1);
        __threadfence();
        if (atomicAdd(sync, 1u) == gridDim.x - 1) {
            *(volatile unsigned *)sync = 0u;
            __threadfence();
            atomicAdd(sync + 1, 1u);
        }
    }
}
__device__ __forceinline__ void grid_wait(unsigned *sync, unsigned gen, unsigned *status, unsigned long long timeout_ns)
{
    if (threadIdx.x == 0) {
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t n = 1;; ++n) {
            unsigned v;
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(sync + 1) : "memory");
            if (v != gen) break;
            if ((n & 63u) == 0 && globaltimer_ns() - t0 > timeout_ns) {
                *(volatile unsigned *)status = 0x201u;
                __threadfence_system();
                break;
            }
        }
        __threadfence();
    }
    __syncthreads();
}

// A float as an unsigned number of the same order, a NaN above all, -0 as 0
__device__ __forceinline__ uint32_t order_key(float v)
{
    if (isnan(v)) return 0xffffffffu;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Eight elements of a row from element h, zeros past H
__device__ __forceinline__ void load8(const void *row, int dtype, int h, int H, bool vec, float (&v)[8])
{
    if (vec && h + 8 <= H) {
        if (dtype == TC_F32) {
            const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(row) + h);
            const float4 x = __ldg(q), y = __ldg(q + 1);
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
        } else {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(row) + h));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint16_t b = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
                v[i] = dtype == TC_BF16 ? __bfloat162float(__ushort_as_bfloat16(b)) : __half2float(__ushort_as_half(b));
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = h + i < H ? load_c(row, h + i, dtype) : 0.0f;
}

// Stage 0: the logits of experts blockIdx.x, + gridDim.x, ...
__device__ void moe_router(const MoeArgs &a, MoeLists &L)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int xt = a.x_bf16 ? TC_BF16 : TC_F16, rs = a.r_dtype == TC_F32 ? 4 : 2;
    const bool x_vec = (reinterpret_cast<uintptr_t>(a.X) & 15u) == 0 && a.ldx % 8 == 0;
    const bool r_vec = (reinterpret_cast<uintptr_t>(a.R) & 15u) == 0 && a.ldr * rs % 16 == 0;
    for (int e = blockIdx.x; e < a.E; e += gridDim.x) {
        const uint8_t *r = static_cast<const uint8_t *>(a.R) + (long long)e * a.ldr * rs;
        for (int t0 = 0; t0 < a.T; t0 += 8) {
            float acc[8] = {};
            for (int h = threadIdx.x * 8; h < a.H; h += MO_THREADS * 8) {
                float rv[8], xv[8];
                load8(r, a.r_dtype, h, a.H, r_vec, rv);
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    if (t0 + t >= a.T) break;
                    load8(static_cast<const uint16_t *>(a.X) + (t0 + t) * a.ldx, xt, h, a.H, x_vec, xv);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[t] = fmaf(rv[i], xv[i], acc[t]);
                }
            }
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                if (t0 + t >= a.T) break;
                acc[t] = warp_sum(acc[t]);
                if (lane == 0) L.red[warp][t] = acc[t];
            }
            __syncthreads();
            if (threadIdx.x < 8 && t0 + (int)threadIdx.x < a.T) {
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < MO_WARPS; ++w) v += L.red[w][threadIdx.x];
                a.logits[(t0 + threadIdx.x) * a.E + e] = v;
            }
            __syncthreads();
        }
    }
}

// The chosen experts of every token, a warp per token: top_k rounds of a
// maximum over the logits' keys, the lowest index among equals.
__device__ void moe_choose(const MoeArgs &a, MoeLists &L)
{
    constexpr int PER = TC_MOE_MAX_EXPERTS / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int t = warp; t < a.T; t += MO_WARPS) {
        uint32_t key[PER];
        float l[PER];
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            key[q] = 0u;
            l[q] = 0.0f;
            if (q * 32 >= a.E) continue;
            if (q * 32 + lane < a.E) {
                l[q] = __ldcg(a.logits + t * a.E + q * 32 + lane);
                key[q] = order_key(l[q]);
            }
        }
        float top = 0.0f, chosen = 0.0f, mine = 0.0f, all = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            uint32_t best = 0u;
            int at = 0x7fffffff;
#pragma unroll
            for (int q = 0; q < PER; ++q) {
                if (q * 32 >= a.E) continue;
                if (key[q] > best) best = key[q], at = q * 32 + lane;      // the lane's lowest index of its largest
            }
            const uint32_t m = __reduce_max_sync(0xffffffffu, best);
            const int e = __reduce_min_sync(0xffffffffu, best == m ? at : 0x7fffffff);
            const float v = m == 0xffffffffu ? __uint_as_float(0x7fc00000u)
                                             : __uint_as_float(m & 0x80000000u ? m & 0x7fffffffu : ~m);
            if (j == 0) {
                top = v;
#pragma unroll
                for (int q = 0; q < PER; ++q) {
                    if (q * 32 >= a.E) continue;
                    if (q * 32 + lane < a.E) all += expf(l[q] - top);
                }
                all = warp_sum(all);
            }
#pragma unroll
            for (int q = 0; q < PER; ++q)
                if (q * 32 + lane == e) key[q] = 0u;
            const float x = expf(v - top);
            chosen += x;
            if (lane == j) {
                mine = x;
                L.id[t * a.k + j] = (uint16_t)e;
                atomicOr(&L.mask[e], 1u << t);
            }
        }
        if (lane < a.k) L.p[t * a.k + lane] = mine / (a.renorm ? chosen : all);
    }
}

// The entries: for each expert with tokens, in index order, its tokens in
// order, 8 to an entry.
__device__ void moe_list(const MoeArgs &a, MoeLists &L)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = tid < a.E ? __popc(L.mask[tid]) : 0, chunks = (n + 7) >> 3;
    uint32_t v = (uint32_t)n << 16 | (uint32_t)chunks, s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += x;
    }
    if (lane == 31) L.scan[warp] = s;
    __syncthreads();
    uint32_t base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < MO_WARPS; ++w) {
        if (w < warp) base += L.scan[w];
        total += L.scan[w];
    }
    s += base - v;                                      // before this expert
    if (tid < a.E) {
        L.off[tid] = (uint16_t)(s >> 16);
        for (int c = 0; c < chunks; ++c) {
            const int i = (int)(s & 0xffffu) + c;
            L.ent_e[i] = (uint16_t)tid;
            L.ent_at[i] = (uint16_t)((s >> 16) + 8 * c);
            L.ent_n[i] = (uint8_t)min(8, n - 8 * c);
        }
    }
    if (tid == 0) L.entries = (int)(total & 0xffffu);
    __syncthreads();
    if (tid < a.T * a.k) {
        const int t = tid / a.k, e = L.id[tid];
        L.pair[L.off[e] + __popc(L.mask[e] & ((1u << t) - 1u))] = (uint16_t)tid;
        if (blockIdx.x == 0) {
            if (a.ids) a.ids[tid] = e;
            if (a.p) a.p[tid] = L.p[tid];
        }
    }
    __syncthreads();
}

template <bool BF16, bool SBF16, int G>
__global__ void __launch_bounds__(MO_THREADS, 1) moe_kernel(const MoeArgs a, const __grid_constant__ MoeMaps maps)
{
    constexpr int GP = Q4_SLAB / G, S = MO_STAGES;
    extern __shared__ uint8_t raw[];
    uint8_t *ring = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    float *space = reinterpret_cast<float *>(ring + MO_RING);       // stage 1: tiles; stage 2: sums
    MoeLists &L = *reinterpret_cast<MoeLists *>(ring + MO_RING + MO_SUMS);
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + MO_RING + MO_SUMS + (sizeof(MoeLists) + 7) / 8 * 8);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t my_ring = smem_u32(ring) + warp * (S * MO_STAGE_BYTES);
    const uint32_t my_bar = smem_u32(bars + warp * S);
    const bool zeros1 = a.w1.zeros != nullptr, zeros2 = a.w2.zeros != nullptr;
    if (lane == 0) {
        prefetch_tmap(&maps.c1);
        prefetch_tmap(&maps.s1);
        prefetch_tmap(&maps.c2);
        prefetch_tmap(&maps.s2);
        for (int i = 0; i < S; ++i) mbar_init(my_bar + 8 * i, 1);
        fence_barrier_init();
    }
    for (int e = threadIdx.x; e < a.E; e += MO_THREADS) L.mask[e] = 0u;

    unsigned gen = 0;
    moe_router(a, L);
    grid_arrive(a.sync, gen);
    grid_wait(a.sync, gen, a.status, a.timeout_ns);
    moe_choose(a, L);
    __syncthreads();
    moe_list(a, L);
    const int entries = L.entries;

    // stage 1: this CTA's units and this warp's share of them
    const int nb = (a.I + 7) / 8;
    const long long units = (long long)entries * nb;
    const long long u0 = blockIdx.x * units / gridDim.x, u1 = (blockIdx.x + 1LL) * units / gridDim.x;
    const int ns1 = (a.H + Q4_SLAB - 1) / Q4_SLAB, ns2 = (a.I + Q4_SLAB - 1) / Q4_SLAB;
    const int wk_n = min(ns1, MO_WARPS), wr_n = MO_WARPS / wk_n;
    const int wr = warp / wk_n, wk = warp - wr * wk_n;
    const bool active = wr < wr_n;
    const int per = active ? (ns1 - wk + wk_n - 1) / wk_n : 0;
    // stage 2: this CTA's rows of hidden, in whole 8s
    const int rows8 = ((a.H + 7) / 8 + (int)gridDim.x - 1) / (int)gridDim.x;
    const int r_lo = min((long long)a.H, (long long)blockIdx.x * rows8 * 8), r_hi = min((long long)a.H, (long long)r_lo + rows8 * 8);
    const int slabs2 = entries * ns2;                   // (entry, slab) pieces, dealt out to the warps

    // lane 0 fetches the warp's pieces: stage 1's, then stage 2's
    long long f_u = active ? u0 + wr : u1;
    int f_s = 0, f_ent = (int)(f_u / nb), f_b = (int)(f_u - (long long)f_ent * nb);
    int f_panel = r_lo, f_i = warp, f_row = r_lo, f_stage = 0, fetched = 0;
    auto piece = [&](const CUtensorMap *c, const CUtensorMap *s, const CUtensorMap *z, int ra, int rb, int slab) {
        const uint32_t st = my_ring + f_stage * MO_STAGE_BYTES, bar = my_bar + 8 * f_stage;
        mbar_arrive_expect_tx(bar, 2 * (1024 + GP * (MOE_SCALE_BOX * 2 + (z ? Q4_ZERO_BOX : 0))));
        tma_load_2d(st, c, bar, slab * (Q4_SLAB / 2), ra);
        tma_load_2d(st + 1024, c, bar, slab * (Q4_SLAB / 2), rb);
        tma_load_2d(st + MO_SCALE_AT, s, bar, ra & ~7, slab * GP);
        tma_load_2d(st + MO_SCALE_AT + 256, s, bar, rb & ~7, slab * GP);
        if (z) {
            tma_load_2d(st + MO_ZERO_AT, z, bar, ra & ~15, slab * GP);
            tma_load_2d(st + MO_ZERO_AT + 256, z, bar, rb & ~15, slab * GP);
        }
        ++fetched;
        if (++f_stage == S) f_stage = 0;
    };
    auto fetch = [&]() {
        if (f_u < u1) {
            const int ra = L.ent_e[f_ent] * 2 * a.I + f_b * 8;
            piece(&maps.c1, &maps.s1, zeros1 ? &maps.z1 : nullptr, ra, ra + a.I, wk + f_s * wk_n);
            if (++f_s == per) {
                f_s = 0;
                f_u += wr_n;
                f_b += wr_n;
                while (f_b >= nb) f_b -= nb, ++f_ent;
            }
        } else if (f_panel < r_hi && f_i < slabs2) {
            const int ent = f_i / ns2, ra = L.ent_e[ent] * a.H + f_row;
            piece(&maps.c2, &maps.s2, zeros2 ? &maps.z2 : nullptr, ra, ra + 8, f_i - ent * ns2);
            f_row += 16;
            if (f_row >= min(r_hi, f_panel + MO_PANEL)) {
                f_row = f_panel;
                f_i += MO_WARPS;
                if (f_i >= slabs2) {
                    f_i = warp;
                    f_panel += MO_PANEL;
                    f_row = f_panel;
                }
            }
        }
    };
    if (lane == 0)
        for (int i = 0; i < S; ++i) fetch();
    __syncwarp();

    const Q4Watch watch{nullptr, a.status, a.timeout_ns};
    const uint32_t word = q4_first_word(g, t);
    int stage = 0, parity = 0;
    bool ok = true;
    auto arrive = [&](int ra, int rb, bool zeros) {      // the next piece, when it is there
        ok = ok && q4_wait(my_bar + 8 * stage, parity, watch);
        __syncwarp();
        const uint8_t *st = ring + (warp * S + stage) * MO_STAGE_BYTES;
        Q4Slab b;
        b.base = st;
        b.codes = word;
        b.s0 = reinterpret_cast<const uint16_t *>(st + MO_SCALE_AT) + (ra & 7) + g;
        b.s1 = reinterpret_cast<const uint16_t *>(st + MO_SCALE_AT + 256) + (rb & 7) + g;
        b.z0 = zeros ? st + MO_ZERO_AT + (ra & 15) + g : nullptr;
        b.z1 = st + MO_ZERO_AT + 256 + (rb & 15) + g;
        return b;
    };
    auto release = [&]() {
        __syncwarp();
        if (lane == 0 && ok) fetch();
        __syncwarp();
        if (++stage == S) stage = 0, parity ^= 1;
    };

    // ------------------------------------------------ stage 1: gate and up
    {
        const uint16_t *X = static_cast<const uint16_t *>(a.X);
        const bool x_vec = (reinterpret_cast<uintptr_t>(X) & 15u) == 0 && (a.ldx & 7) == 0;
        uint32_t xf[1][8][4];
        int have_ent = -1, have_slab = -1;
        int ent = active ? (int)((u0 + wr) / nb) : 0, b8 = active ? (int)((u0 + wr) - (long long)ent * nb) : 0;
        for (long long first = u0 + wr; active && first < u1; first += MO_HOLD * wr_n) {
            int held = 0;
            for (long long u = first; u < u1 && held < MO_HOLD; u += wr_n, ++held) {
                float acc[1][4] = {};
                const int ra = L.ent_e[ent] * 2 * a.I + b8 * 8;
                for (int s = 0; s < per; ++s) {
                    const int slab = wk + s * wk_n;
                    if (ent != have_ent || slab != have_slab) {
                        have_ent = ent, have_slab = slab;
#pragma unroll
                        for (int j = 0; j < 8; ++j) xf[0][j][0] = xf[0][j][1] = xf[0][j][2] = xf[0][j][3] = 0u;
                        if (g < L.ent_n[ent]) {
                            const uint16_t *row = X + (L.pair[L.ent_at[ent] + g] / a.k) * a.ldx;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const uint4 v = q4_load_x(row, slab * Q4_SLAB + 32 * j + 8 * t, a.H, x_vec);
                                xf[0][j][0] = v.x, xf[0][j][1] = v.y, xf[0][j][2] = v.z, xf[0][j][3] = v.w;
                            }
                        }
                    }
                    const Q4Slab b = arrive(ra, ra + a.I, zeros1);
                    q4_slab<BF16, SBF16, 1, G, MOE_SCALE_BOX>(acc, b, xf);
                    release();
                }
                float *tile = space + (held * MO_WARPS + warp) * MO_TILE + 2 * t * MO_TILE_LD + g;
#pragma unroll
                for (int e = 0; e < 4; ++e) tile[(e & 1) * MO_TILE_LD + 8 * (e >> 1)] = acc[0][e];
                b8 += wr_n;
                while (b8 >= nb) b8 -= nb, ++ent;
            }
            __syncwarp();
            q4_group_sync(wr, wk_n);
            // two threads per token and four rows: each adds every other
            // warp's tile, in warp order, then the two join
            const int half = lane & 1;
            for (int e = (wk * 32 + lane) >> 1; e < MO_HOLD * 16; e += wk_n * 16) {
                const int hu = e >> 4, c = (e >> 1) & 7, r = (e & 1) * 4;
                const long long u = first + (long long)hu * wr_n;
                const int ue = hu < held ? (int)(u / nb) : 0;
                const bool in = hu < held && c < L.ent_n[ue];
                const float *p = space + (hu * MO_WARPS + warp - wk) * MO_TILE + c * MO_TILE_LD + r;
                float v[8] = {};
#pragma unroll
                for (int w = 0; w < MO_WARPS; w += 2)
                    if (in && w + half < wk_n) {
                        const float4 x = *reinterpret_cast<const float4 *>(p + (w + half) * MO_TILE);
                        const float4 y = *reinterpret_cast<const float4 *>(p + (w + half) * MO_TILE + 8);
                        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
                        v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
                    }
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 1);
                if (!in) continue;
                const int i0 = (int)(u - (long long)ue * nb) * 8 + r + 2 * half;
                uint16_t *h = a.h + L.pair[L.ent_at[ue] + c] * a.ldh + i0;
                uint16_t hi[2], lo[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float gt = half ? v[2 + i] : v[i], up = half ? v[6 + i] : v[4 + i];
                    const float x = gt / (1.0f + expf(-gt)) * up;
                    const __nv_bfloat16 b = __float2bfloat16_rn(x);
                    const float rest = x - __bfloat162float(b);
                    hi[i] = __bfloat16_as_ushort(b);
                    // (an infinity or a NaN stands in the first part alone)
                    lo[i] = __bfloat16_as_ushort(__float2bfloat16_rn(isfinite(rest) ? rest : 0.0f));
                    if (i0 + i >= a.I) hi[i] = lo[i] = 0;
                }
                // (ldh is I rounded up to 8, so both elements are in the row)
                *reinterpret_cast<uint32_t *>(h) = hi[0] | (uint32_t)hi[1] << 16;
                *reinterpret_cast<uint32_t *>(h + (long long)a.T * a.k * a.ldh) = lo[0] | (uint32_t)lo[1] << 16;
            }
            q4_group_sync(wr, wk_n);          // the tiles are read before the next ones are written
        }
    }
    grid_arrive(a.sync, gen);
    // this warp's sums start at zero while the others arrive
    float *sums = space + warp * a.T * MO_PANEL;
    for (int i = lane; i < a.T * MO_PANEL; i += 32) sums[i] = 0.0f;
    grid_wait(a.sync, gen, a.status, a.timeout_ns);

    // ------------------------------------------------ stage 2: down
    for (int panel = r_lo; panel < r_hi; panel += MO_PANEL) {
        const int p_hi = min(r_hi, panel + MO_PANEL);
        for (int i = warp; i < slabs2; i += MO_WARPS) {
            const int ent = i / ns2, slab = i - ent * ns2, n = L.ent_n[ent], at = L.ent_at[ent];
            uint32_t xf[2][8][4];
            {
                const uint16_t *row = a.h + (long long)(g < n ? L.pair[at + g] : 0) * a.ldh;
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int k = slab * Q4_SLAB + 32 * j + 8 * t;
                        uint4 v = make_uint4(0u, 0u, 0u, 0u);
                        if (g < n && k < a.I)
                            v = __ldcg(reinterpret_cast<const uint4 *>(row + (long long)q * a.T * a.k * a.ldh + k));
                        xf[q][j][0] = v.x, xf[q][j][1] = v.y, xf[q][j][2] = v.z, xf[q][j][3] = v.w;
                    }
            }
            // the columns' tokens and weights (columns 2 t and 2 t + 1)
            int tok[2];
            float pw[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int pr = 2 * t + c < n ? L.pair[at + 2 * t + c] : 0;
                tok[c] = 2 * t + c < n ? pr / a.k : -1;
                pw[c] = L.p[pr];
            }
            for (int row = panel; row < p_hi; row += 16) {
                float acc[1][4] = {};
                const int ra = L.ent_e[ent] * a.H + row;
                const Q4Slab b = arrive(ra, ra + 8, zeros2);
                q4_slab<true, SBF16, 2, G, MOE_SCALE_BOX, true>(acc, b, xf);
                release();
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (tok[c] >= 0) {
                        float *y = sums + tok[c] * MO_PANEL + (row - panel) + g;
                        y[0] = fmaf(pw[c], acc[0][c], y[0]);
                        y[8] = fmaf(pw[c], acc[0][2 + c], y[8]);
                    }
                __syncwarp();
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < a.T * MO_PANEL; i += MO_THREADS) {
            const int tk = i / MO_PANEL, r = i - tk * MO_PANEL;
            float y = 0.0f;
#pragma unroll
            for (int w = 0; w < MO_WARPS; ++w) {
                y += space[w * a.T * MO_PANEL + i];
                space[w * a.T * MO_PANEL + i] = 0.0f;
            }
            if (panel + r < p_hi) store_c1(a.Y, tk * a.ldy + panel + r, y, a.y_dtype);
        }
        __syncthreads();
    }
    // after an expired wait: copies still in flight land (within a limit)
    // before shared memory is released
    if (!ok && lane == 0)
        for (int i = 0; i < S; ++i) {
            const int n = (fetched + S - 1 - i) / S;
            if (n > 0) q4_drain(my_bar + 8 * i, (uint32_t)(n - 1) & 1u);
        }
}

template <bool BF16, bool SBF16, int G>
cudaError_t launch_one(const MoeArgs &a, const MoeMaps &m, int grid, cudaStream_t st)
{
    constexpr auto kern = moe_kernel<BF16, SBF16, G>;
    static std::atomic<bool> configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, MO_SMEM);
        if (e != cudaSuccess) return e;
        configured[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(MO_THREADS);
    cfg.dynamicSmemBytes = MO_SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, m);
}

template <bool BF16, bool SBF16>
cudaError_t launch_group(const MoeArgs &a, const MoeMaps &m, int grid, cudaStream_t st)
{
    switch (a.w1.group) {
    case 32: return launch_one<BF16, SBF16, 32>(a, m, grid, st);
    case 64: return launch_one<BF16, SBF16, 64>(a, m, grid, st);
    default: return launch_one<BF16, SBF16, 128>(a, m, grid, st);
    }
}

}  // namespace

cudaError_t launch_moe(const MoeArgs &a, const MoeMaps &m, int grid, cudaStream_t st)
{
    if (a.x_bf16) return a.w1.scale_bf16 ? launch_group<true, true>(a, m, grid, st) : launch_group<true, false>(a, m, grid, st);
    return a.w1.scale_bf16 ? launch_group<false, true>(a, m, grid, st) : launch_group<false, false>(a, m, grid, st);
}

}  // namespace tc
