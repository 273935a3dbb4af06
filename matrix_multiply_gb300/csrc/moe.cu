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
// is kept as a sum of bf16 parts, multiplied one after the other: two of them
// (16 bits of significand, any exponent) where y has 16 bits, 11 of them
// significant at most (of 2048 bf16 outputs of one token 9 are not the nearest to
// their 64-bit values, of the same formulas in fp32 4); three (all 24 bits) where
// y is fp32.  Deterministic: lists in index order, sums in fixed orders.
//
// Measured: 1 token, hidden 2048, inter 768, 8 of 64 experts, groups of 128:
// 18.4 us for 20.0 MB, of which the launch takes 3.1, each stage's dependent
// loads, barriers and first passes through its code the rest.  16 tokens,
// hidden 4096, inter 1408, 8 of 64, groups of 64 with zero points: 174 us for
// about 535 MB, 46% of a plain copy's rate, bound by issue and the fixed
// latencies of the widening chain (about 460 instructions per 16 rows x 256 k;
// schedulers issue in 56% of the cycles), with pieces of 16 rows 186.  As separate launches the stages
// would add two of them, with their drains, to every call.
#include "q4.cuh"

#include <atomic>

namespace tc {
namespace {

constexpr int MO_WARPS = 16, MO_THREADS = MO_WARPS * 32;
constexpr int MO_TILE_LD = 20, MO_TILE = 8 * MO_TILE_LD; // floats: a unit's partial tile, 8 tokens x 16 rows
constexpr int MO_PANEL = 32;                             // rows of hidden per stage-2 panel, at most
constexpr int MO_PAIRS = TC_MOE_MAX_TOKENS * TC_MOE_MAX_TOPK;
// Shared memory: the rings (the codes of all warps, then their scales and
// zero points) and the sums, stage 1's tiles or stage 2's panel.  A piece of
// a ring is one unit of stage 1 or 16 rows of stage 2; TALL two units, 32 rows.
template <int G, bool TALL>
struct MoSpace {
    static constexpr int GP = Q4_SLAB / G;
    static constexpr int STAGES = TALL ? 2 : 3, ROWS = TALL ? 32 : 16, CODES = ROWS * 128;
    static constexpr int SCALE2_BOX = 8 + ROWS, ZERO2_BOX = 16 + ROWS;
    static constexpr int up128(int x) { return (x + 127) / 128 * 128; }
    static constexpr int larger(int x, int y) { return x > y ? x : y; }
    // stage 1: two parts of GP groups' scales (zero points), on 128 bytes where they are copied apart
    static constexpr int S_PART = up128(GP * MOE_SCALE_BOX * 2), Z_PART = up128(GP * Q4_ZERO_BOX);
    static constexpr int ZERO_AT = up128(larger(2 * S_PART, GP * SCALE2_BOX * 2));
    static constexpr int SIDE = ZERO_AT + up128(larger(2 * Z_PART, GP * ZERO2_BOX));
    static constexpr int RING = MO_WARPS * STAGES * (CODES + SIDE);
    static constexpr int HOLD = TALL && G == 32 ? 4 : 6;     // units whose partial tiles are held before they are added
    static constexpr int SUMS = MO_WARPS * (TALL ? moe_panel_tokens(G) : TC_MOE_MAX_TOKENS) * MO_PANEL * 4;
    static_assert(HOLD * MO_WARPS * MO_TILE * 4 <= SUMS, "stage 1's tiles share stage 2's space");
    static_assert(TC_MOE_MAX_TOKENS * 16 <= moe_panel_tokens(G) * MO_PANEL, "a panel of 16 rows fits for any tokens");
};
static_assert(MO_PAIRS <= MO_THREADS && TC_MOE_MAX_EXPERTS <= MO_THREADS && TC_MOE_MAX_TOKENS <= 32, "one thread each");

struct MoeLists {
    uint32_t mask[TC_MOE_MAX_EXPERTS];       // tokens that chose the expert
    uint16_t off[TC_MOE_MAX_EXPERTS];        // the expert's first place in `pair`
    uint16_t pair[MO_PAIRS];                 // t * top_k + j, by expert, then token
    uint16_t id[MO_PAIRS];                   // of pair t * top_k + j: the expert
    float p[MO_PAIRS];                       //   and its weight
    uint16_t ent_e[MO_PAIRS], ent_at[MO_PAIRS];   // entries: expert, first place in `pair`
    uint8_t ent_n[MO_PAIRS];                      //   and number of tokens (1 .. 8)
    uint8_t tok[MO_PAIRS];                        // the token of pair[i]
    int entries;
    float red[MO_WARPS][8];
};
template <int G, bool TALL>
constexpr int MO_SMEM = 1024 + MoSpace<G, TALL>::RING + MoSpace<G, TALL>::SUMS + (int)sizeof(MoeLists) +
                        MO_WARPS * MoSpace<G, TALL>::STAGES * 8 + 16;
static_assert(MO_SMEM<32, true> <= SMEM_LIMIT && MO_SMEM<64, true> <= SMEM_LIMIT && MO_SMEM<128, true> <= SMEM_LIMIT &&
                  MO_SMEM<32, false> <= SMEM_LIMIT,
              "one CTA per SM");

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// All CTAs of the grid (a cooperative launch: all are resident).  One word
// counts arrivals: what the CTAs add makes 2^31 together, so its top bit
// flips when the last has arrived, and it needs no reset.  The wait is
// bounded: past the limit the kernel reports and goes on, its outputs
// undefined.
__device__ __forceinline__ unsigned grid_arrive(unsigned *sync, bool drop = false)
{
    unsigned old = 0;
    __syncthreads();
    if (threadIdx.x == 0 && !drop) {
        const unsigned add = blockIdx.x == 0 ? 0x80000000u - (gridDim.x - 1) : 1u;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(sync), "r"(add) : "memory");
    }
    return old;
}
__device__ __forceinline__ void grid_wait(unsigned *sync, unsigned old, unsigned *status, unsigned long long timeout_ns)
{
    if (threadIdx.x == 0) {
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t n = 1;; ++n) {
            unsigned v;
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(sync) : "memory");
            if ((v ^ old) & 0x80000000u) break;
            if ((n & 63u) == 0 && globaltimer_ns() - t0 > timeout_ns) {
                *(volatile unsigned *)status = 0x201u;
                __threadfence_system();
                break;
            }
        }
    }
    __syncthreads();
}

// A float as an unsigned number of the same order, a NaN above all, -0 as 0;
// and back
__device__ __forceinline__ uint32_t order_key(float v)
{
    if (isnan(v)) return 0xffffffffu;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return k == 0xffffffffu ? __uint_as_float(0x7fc00000u) : __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// the low or high half of a register as fp32
template <bool BF16>
__device__ __forceinline__ float half_word(uint32_t w, int high)
{
    if constexpr (BF16) return __uint_as_float(high ? w & 0xffff0000u : w << 16);
    return __half2float(__ushort_as_half((unsigned short)(high ? w >> 16 : w)));
}

// Stage 0: the logits of (expert, up to TW tokens) tasks blockIdx.x, +
// gridDim.x, ...; a thread takes eight elements of the rows at a time, all of
// a step's loads issued before their use.
template <bool BF16, int TW>
__device__ __forceinline__ void moe_router(const MoeArgs &a, MoeLists &L)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool rf32 = a.r_dtype == TC_F32;
    const bool x_vec = (reinterpret_cast<uintptr_t>(a.X) & 15u) == 0 && a.ldx % 8 == 0;
    const bool r_vec = (reinterpret_cast<uintptr_t>(a.R) & 15u) == 0 && a.ldr % (rf32 ? 4 : 8) == 0;
    const int chunks = (a.T + TW - 1) / TW;
    for (int task = blockIdx.x; task < a.E * chunks; task += gridDim.x) {
        const int e = task / chunks, t0 = (task - e * chunks) * TW;
        float acc[TW] = {};
        for (int h = threadIdx.x * 8; h < a.H; h += MO_THREADS * 8) {
            uint4 x[TW];
            float r[8];
#pragma unroll
            for (int t = 0; t < TW; ++t)
                x[t] = q4_load_x(static_cast<const uint16_t *>(a.X) + min(t0 + t, a.T - 1) * a.ldx, h, a.H, x_vec);
            if (rf32) {
                const float *row = static_cast<const float *>(a.R) + e * a.ldr + h;
                if (r_vec && h + 8 <= a.H) {
                    const float4 u = __ldg(reinterpret_cast<const float4 *>(row)), v = __ldg(reinterpret_cast<const float4 *>(row) + 1);
                    r[0] = u.x, r[1] = u.y, r[2] = u.z, r[3] = u.w, r[4] = v.x, r[5] = v.y, r[6] = v.z, r[7] = v.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) r[i] = h + i < a.H ? row[i] : 0.0f;
                }
            } else {
                const uint4 v = q4_load_x(static_cast<const uint16_t *>(a.R) + e * a.ldr, h, a.H, r_vec);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) r[i] = half_word<BF16>(w[i >> 1], i & 1);
            }
#pragma unroll
            for (int t = 0; t < TW; ++t) {
                const uint32_t w[4] = {x[t].x, x[t].y, x[t].z, x[t].w};
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[t] = fmaf(r[i], half_word<BF16>(w[i >> 1], i & 1), acc[t]);
            }
        }
        // the warp's sums: halving the tokens a lane holds, then the lanes
        int tok = 0;
#pragma unroll
        for (int n = TW / 2, o = 16; n >= 1; n >>= 1, o >>= 1) {
            const bool up = lane & o;
            if (up) tok += n;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float keep = up ? acc[i + n] : acc[i], send = up ? acc[i] : acc[i + n];
                acc[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
        }
#pragma unroll
        for (int o = 16 / TW; o > 0; o >>= 1) acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
        if ((lane & (32 / TW - 1)) == 0) L.red[warp][tok] = acc[0];
        __syncthreads();
        if (threadIdx.x < TW && t0 + (int)threadIdx.x < a.T) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < MO_WARPS; ++w) v += L.red[w][threadIdx.x];
            a.logits[(t0 + threadIdx.x) * a.E + e] = v;
        }
        __syncthreads();
    }
}

// The chosen experts of every token: a warp per token, top_k rounds of a
// maximum over the logits' keys (NQ per lane), the lowest index among equals.
template <int NQ>
__device__ __forceinline__ void moe_choose(const MoeArgs &a, MoeLists &L)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int t = warp; t < a.T; t += MO_WARPS) {
        uint32_t key[NQ];
        float l[NQ];
#pragma unroll
        for (int q = 0; q < NQ; ++q) l[q] = q * 32 + lane < a.E ? __ldcg(a.logits + t * a.E + q * 32 + lane) : 0.0f;
#pragma unroll
        for (int q = 0; q < NQ; ++q) key[q] = q * 32 + lane < a.E ? order_key(l[q]) : 0u;
        uint32_t top = 0u, mine = 0u, id = 0u;
#pragma unroll 1
        for (int j = 0; j < a.k; ++j) {
            uint32_t best = key[0];
            int at = lane;
#pragma unroll
            for (int q = 1; q < NQ; ++q)
                if (key[q] > best) best = key[q], at = q * 32 + lane;      // the lane's lowest index of its largest
            const uint32_t m = __reduce_max_sync(0xffffffffu, best);
            const uint32_t e = __reduce_min_sync(0xffffffffu, best == m ? (uint32_t)at : 0xffffffffu);
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                if (q * 32 + lane == (int)e) key[q] = 0u;
            if (j == 0) top = m;
            if (lane == j) mine = m, id = e;
        }
        if (lane < a.k) {
            L.id[t * a.k + lane] = (uint16_t)id;
            atomicOr(&L.mask[id], 1u << t);
        }
        const float ftop = key_value(top), x = lane < a.k ? expf(key_value(mine) - ftop) : 0.0f;
        float sum = x;
        if (!a.renorm) {
            sum = 0.0f;
#pragma unroll
            for (int q = 0; q < NQ; ++q) sum += q * 32 + lane < a.E ? expf(l[q] - ftop) : 0.0f;
        }
        sum = warp_sum(sum);
        if (lane < a.k) L.p[t * a.k + lane] = x / sum;
    }
}

// The entries: for each expert with tokens, in index order, its tokens in
// order, 8 to an entry.  One warp: its lanes scan 32 experts at a time.
__device__ __forceinline__ void moe_list(const MoeArgs &a, MoeLists &L)
{
    const int lane = threadIdx.x & 31;
    uint32_t base = 0;                                  // places in `pair` << 16 | entries so far
    for (int e0 = 0; e0 < a.E; e0 += 32) {
        const int e = e0 + lane, n = e < a.E ? __popc(L.mask[e]) : 0, chunks = (n + 7) >> 3;
        const uint32_t v = (uint32_t)n << 16 | (uint32_t)chunks;
        uint32_t s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += x;
        }
        const uint32_t at = base + s - v;
        base += __shfl_sync(0xffffffffu, s, 31);
        if (n > 0) L.off[e] = (uint16_t)(at >> 16);
        for (int c = 0; c < chunks; ++c) {
            const int i = (int)(at & 0xffffu) + c;
            L.ent_e[i] = (uint16_t)e;
            L.ent_at[i] = (uint16_t)((at >> 16) + 8 * c);
            L.ent_n[i] = (uint8_t)min(8, n - 8 * c);
        }
    }
    if (lane == 0) L.entries = (int)(base & 0xffffu);
    __syncwarp();
    for (int i = lane; i < a.T * a.k; i += 32) {
        const int t = (int)((unsigned)i / (unsigned)a.k), e = L.id[i];
        L.pair[L.off[e] + __popc(L.mask[e] & ((1u << t) - 1u))] = (uint16_t)i;
        L.tok[L.off[e] + __popc(L.mask[e] & ((1u << t) - 1u))] = (uint8_t)t;
    }
}

template <bool BF16, bool SBF16, int G, int PARTS, bool TALL>
__global__ void __launch_bounds__(MO_THREADS, 1) moe_kernel(const MoeArgs a, const __grid_constant__ MoeMaps maps)
{
    using Space = MoSpace<G, TALL>;
    constexpr int GP = Space::GP, S = Space::STAGES, HOLD = Space::HOLD, W = TALL ? 2 : 1;
    extern __shared__ uint8_t raw[];
    uint8_t *ring = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint8_t *side = ring + MO_WARPS * S * Space::CODES;
    float *space = reinterpret_cast<float *>(ring + Space::RING);   // stage 1: tiles; stage 2: sums
    MoeLists &L = *reinterpret_cast<MoeLists *>(ring + Space::RING + Space::SUMS);
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + Space::RING + Space::SUMS + (sizeof(MoeLists) + 7) / 8 * 8);

    const int warp = uniform_warp(), lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t my_ring = smem_u32(ring) + warp * (S * Space::CODES), my_side = smem_u32(side) + warp * (S * Space::SIDE);
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
    __syncwarp();
    for (int e = threadIdx.x; e < a.E; e += MO_THREADS) L.mask[e] = 0u;

    if (a.T <= 2)
        moe_router<BF16, 2>(a, L);
    else
        moe_router<BF16, 8>(a, L);
    unsigned old = grid_arrive(a.sync, a.debug_drop == 1 && blockIdx.x == 1);

    // what does not depend on the choice, while the others arrive
    const int G1 = (int)gridDim.x, nb = (a.I + 7) >> 3, nbp = (nb + W - 1) / W;      // units and pieces per entry
    const int ns1 = (a.H + Q4_SLAB - 1) / Q4_SLAB, ns2 = (a.I + Q4_SLAB - 1) / Q4_SLAB;
    int wk_n = MO_WARPS, wr_n = 1, wr = 0, wk = warp;              // stage 1: warps along hidden, groups along the units
    if (ns1 < MO_WARPS) {
        wk_n = ns1;
        wr_n = (unsigned)MO_WARPS / (unsigned)ns1;
        wr = (unsigned)warp / (unsigned)ns1;
        wk = warp - wr * ns1;
    }
    const bool active = wr < wr_n;
    const int per = !active ? 0 : ns1 <= MO_WARPS ? 1 : (ns1 - wk + MO_WARPS - 1) / MO_WARPS;
    // stage 2: this CTA's rows of hidden, in whole 8s
    const int r_lo = (int)min((long long)a.H, (long long)blockIdx.x * a.rows8 * 8);
    const int r_hi = (int)min((long long)a.H, (long long)r_lo + a.rows8 * 8);
    // bytes between the two 8-row parts' scales and zero points in stage 1
    const int s_part = maps.s1_3d ? GP * MOE_SCALE_BOX * 2 : Space::S_PART, z_part = maps.z1_3d ? GP * Q4_ZERO_BOX : Space::Z_PART;

    grid_wait(a.sync, old, a.status, a.timeout_ns);
    if (a.E <= 32)
        moe_choose<1>(a, L);
    else if (a.E <= 64)
        moe_choose<2>(a, L);
    else if (a.E <= 128)
        moe_choose<4>(a, L);
    else if (a.E <= 256)
        moe_choose<8>(a, L);
    else
        moe_choose<16>(a, L);
    __syncthreads();
    if (warp == 0) moe_list(a, L);
    __syncthreads();
    const int entries = L.entries;
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x < a.T * a.k) {
        if (a.ids) a.ids[threadIdx.x] = L.id[threadIdx.x];
        if (a.p) a.p[threadIdx.x] = L.p[threadIdx.x];
    }

    // stage 1: an equal share of the pieces for every CTA
    const unsigned units = (unsigned)entries * (unsigned)nbp, share = units / (unsigned)G1, extra = units - share * G1;
    const unsigned u0 = blockIdx.x * share + min(blockIdx.x, extra), u1 = u0 + share + (blockIdx.x < extra ? 1u : 0u);
    const int slabs2 = entries * ns2;                   // stage 2's (entry, slab) pieces, dealt out to the warps
    const unsigned u_first = active ? u0 + wr : u1;
    const int ent_first = (int)(u_first / (unsigned)nbp), b_first = (int)(u_first - (unsigned)ent_first * nbp);

    // fetching the warp's pieces: stage 1's, then stage 2's
    unsigned f_u = u_first;
    int f_s = 0, f_ent = ent_first, f_b = b_first, f_panel = r_lo, f_i = warp, f_row = 0, f_stage = 0, fetched = 0;
    uint32_t bytes1 = W * 2048 + 2 * GP * MOE_SCALE_BOX * 2 + (zeros1 ? 2 * GP * Q4_ZERO_BOX : 0);
    if (a.debug_drop == 2 && blockIdx.x == 0) bytes1 += 16;
    const uint32_t bytes2 = min(a.panel, Space::ROWS) * 128 + GP * Space::SCALE2_BOX * 2 + (zeros2 ? GP * Space::ZERO2_BOX : 0);
    const uint32_t leader = elect_one();
    auto fetch = [&]() {                                // the whole warp
        const uint32_t st = my_ring + f_stage * Space::CODES, sd = my_side + f_stage * Space::SIDE, bar = my_bar + 8 * f_stage;
        if (f_u < u1) {
            const int half = L.ent_e[f_ent] * 2, slab = wk + f_s * MO_WARPS, x = f_b * W * 8;
            arrive_expect_by(bar, bytes1, leader);
            tma_load_3d_by(st, &maps.c1, bar, slab * (Q4_SLAB / 2), x, half, leader);
            if (W == 2) tma_load_3d_by(st + 2048, &maps.c1, bar, slab * (Q4_SLAB / 2), x + 8, half, leader);
            const int ra = half * a.I + x, rb = ra + a.I;
            if (maps.s1_3d) {
                tma_load_3d_by(sd, &maps.s1, bar, x, slab * GP, half, leader);
            } else {
                tma_load_2d_by(sd, &maps.s1, bar, ra & ~7, slab * GP, leader);
                tma_load_2d_by(sd + Space::S_PART, &maps.s1, bar, rb & ~7, slab * GP, leader);
            }
            if (zeros1) {
                if (maps.z1_3d) {
                    tma_load_3d_by(sd + Space::ZERO_AT, &maps.z1, bar, x & ~15, slab * GP, half, leader);
                } else {
                    tma_load_2d_by(sd + Space::ZERO_AT, &maps.z1, bar, ra & ~15, slab * GP, leader);
                    tma_load_2d_by(sd + Space::ZERO_AT + Space::Z_PART, &maps.z1, bar, rb & ~15, slab * GP, leader);
                }
            }
            if (++f_s == per) {
                f_s = 0;
                f_u += wr_n;
                f_b += wr_n;
                while (f_b >= nbp) f_b -= nbp, ++f_ent;
            }
        } else if (f_panel < r_hi && f_i < slabs2) {
            const int ent = ns2 == 1 ? f_i : (int)((unsigned)f_i / (unsigned)ns2), slab = f_i - ent * ns2;
            const int row = L.ent_e[ent] * a.H + f_panel + f_row;
            arrive_expect_by(bar, bytes2, leader);
            tma_load_2d_by(st, &maps.c2, bar, slab * (Q4_SLAB / 2), row, leader);
            tma_load_2d_by(sd, &maps.s2, bar, row & ~7, slab * GP, leader);
            if (zeros2) tma_load_2d_by(sd + Space::ZERO_AT, &maps.z2, bar, row & ~15, slab * GP, leader);
            f_row += Space::ROWS;
            if (f_row >= min(r_hi - f_panel, a.panel)) {
                f_row = 0;
                f_i += MO_WARPS;
                if (f_i >= slabs2) f_i = warp, f_panel += a.panel;
            }
        } else {
            return;
        }
        ++fetched;
        if (++f_stage == S) f_stage = 0;
    };
#pragma unroll 1
    for (int i = 0; i < S; ++i) fetch();

    const Q4Watch watch{nullptr, a.status, a.timeout_ns};
    const uint32_t word = q4_first_word(g, t);
    int stage = 0, parity = 0;
    bool ok = true;
    auto arrive = [&]() {                                // the next piece, when it is there
        ok = ok && q4_wait(my_bar + 8 * stage, parity, watch);
        __syncwarp();
    };
    auto codes_at = [&]() { return ring + (warp * S + stage) * Space::CODES; };
    auto side_at = [&]() { return side + (warp * S + stage) * Space::SIDE; };
    auto release = [&]() {
        __syncwarp();
        if (__all_sync(0xffffffffu, ok)) fetch();
        if (++stage == S) stage = 0, parity ^= 1;
    };

    // ------------------------------------------------ stage 1: gate and up
    {
        const uint16_t *X = static_cast<const uint16_t *>(a.X);
        const bool x_vec = (reinterpret_cast<uintptr_t>(X) & 15u) == 0 && (a.ldx & 7) == 0;
        uint32_t xf[1][8][4];
        int have_ent = -1, have_slab = -1;
        int ent = ent_first, b8 = b_first;
        constexpr int hold = HOLD / W;                           // pieces
        for (unsigned first = u_first; first < u1; first += hold * wr_n) {
            int held = 0;
            for (unsigned u = first; u < u1 && held < hold; u += wr_n, ++held) {
                float acc[W][1][4] = {};
                const int i8 = b8 * W * 8, ra = L.ent_e[ent] * 2 * a.I + i8, rb = ra + a.I;
                // where the parts' first rows lie in their copies
                const int sa = maps.s1_3d ? 0 : ra & 7, sb = maps.s1_3d ? 0 : rb & 7;
                const int za = maps.z1_3d ? i8 & 15 : ra & 15, zb = maps.z1_3d ? i8 & 15 : rb & 15;
                for (int s = 0; s < per; ++s) {
                    const int slab = wk + s * MO_WARPS;
                    if (ent != have_ent || slab != have_slab) {
                        have_ent = ent, have_slab = slab;
#pragma unroll
                        for (int j = 0; j < 8; ++j) xf[0][j][0] = xf[0][j][1] = xf[0][j][2] = xf[0][j][3] = 0u;
                        if (g < L.ent_n[ent]) {
                            const uint16_t *row = X + L.tok[L.ent_at[ent] + g] * a.ldx;
                            q4_load_slab<false>(xf[0], row, (long long)slab * Q4_SLAB + 8 * t, a.H, x_vec && slab < a.H / Q4_SLAB);
                        }
                    }
                    arrive();
                    const uint8_t *sd = side_at();
                    Q4Slab b;
                    b.base = codes_at();
                    b.codes = word;
                    b.s0 = reinterpret_cast<const uint16_t *>(sd) + sa + g;
                    b.s1 = reinterpret_cast<const uint16_t *>(sd + s_part) + sb + g;
                    b.z0 = zeros1 ? sd + Space::ZERO_AT + za + g : nullptr;
                    b.z1 = sd + Space::ZERO_AT + z_part + zb + g;
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        q4_slab<BF16, SBF16, 1, G, MOE_SCALE_BOX>(acc[i], b, xf);
                        b.base += 2048, b.s0 += 8, b.s1 += 8, b.z1 += 8;
                        if (zeros1) b.z0 += 8;
                    }
                    release();
                }
                float *tile = space + (held * W * MO_WARPS + warp) * MO_TILE + 2 * t * MO_TILE_LD + g;
#pragma unroll
                for (int i = 0; i < W; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        tile[i * MO_WARPS * MO_TILE + (e & 1) * MO_TILE_LD + 8 * (e >> 1)] = acc[i][0][e];
                b8 += wr_n;
                while (b8 >= nbp) b8 -= nbp, ++ent;
            }
            __syncwarp();
            q4_group_sync(wr, wk_n);
            // two threads per token and four rows: each adds every other
            // warp's tile, in warp order, then the two join
            const int half = lane & 1;
            for (int e = (wk * 32 + lane) >> 1; e < HOLD * 16; e += wk_n * 16) {
                const int hu = e >> 4, hp = hu / W, c = (e >> 1) & 7, r = (e & 1) * 4;
                const unsigned u = first + (unsigned)(hp * wr_n);
                const int ue = hp < held ? (int)(u / (unsigned)nbp) : 0;
                const int ub = (int)(u - (unsigned)ue * nbp) * W + (hu - hp * W);       // the unit within the entry
                const bool in = hp < held && ub < nb && c < L.ent_n[ue];
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
                const int i0 = ub * 8 + r + 2 * half;
                uint16_t *h = a.h + L.pair[L.ent_at[ue] + c] * a.ldh + i0;
                uint32_t part[PARTS] = {};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float gt = q4_whole<BF16>(half ? v[2 + i] : v[i]), up = q4_whole<BF16>(half ? v[6 + i] : v[4 + i]);
                    float x = i0 + i < a.I ? gt / (1.0f + expf(-gt)) * up : 0.0f;
#pragma unroll
                    for (int q = 0; q < PARTS; ++q) {
                        const __nv_bfloat16 b = __float2bfloat16_rn(x);
                        part[q] |= (uint32_t)__bfloat16_as_ushort(b) << (16 * i);
                        x -= __bfloat162float(b);
                        if (!isfinite(x)) x = 0.0f;            // an infinity or a NaN stands in the first part alone
                    }
                }
                // (ldh is I rounded up to 8, so both elements are in the row)
#pragma unroll
                for (int q = 0; q < PARTS; ++q)
                    *reinterpret_cast<uint32_t *>(h + (long long)q * a.T * a.k * a.ldh) = part[q];
            }
            q4_group_sync(wr, wk_n);          // the tiles are read before the next ones are written
        }
    }
    old = grid_arrive(a.sync);
    // this warp's sums start at zero while the others arrive
    const int pld = TALL && a.T > moe_panel_tokens(G) ? 16 : MO_PANEL;      // a token's sums of a panel
    float *sums = space + warp * a.T * pld;
    for (int i = lane; i < a.T * pld; i += 32) sums[i] = 0.0f;
    grid_wait(a.sync, old, a.status, a.timeout_ns);

    // ------------------------------------------------ stage 2: down
    for (int panel = r_lo; panel < r_hi; panel += a.panel) {
        const int p_hi = min(r_hi, panel + a.panel);
        for (int i = warp; i < slabs2; i += MO_WARPS) {
            const int ent = (int)((unsigned)i / (unsigned)ns2), slab = i - ent * ns2, n = L.ent_n[ent], at = L.ent_at[ent];
            uint32_t xf[PARTS][8][4];
            {
                const uint16_t *row = a.h + (long long)(g < n ? L.pair[at + g] : 0) * a.ldh;
#pragma unroll
                for (int q = 0; q < PARTS; ++q)
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
                tok[c] = 2 * t + c < n ? L.tok[at + 2 * t + c] : -1;
                pw[c] = 2 * t + c < n ? q4_whole<true>(L.p[L.pair[at + 2 * t + c]]) : 0.0f;   // (h is bf16)
            }
            for (int row0 = 0; row0 < p_hi - panel; row0 += Space::ROWS) {
                constexpr int HALVES = Space::ROWS / 16;
                float acc[HALVES][1][4] = {};
                const int ra = L.ent_e[ent] * a.H + panel + row0;
                arrive();
                const uint8_t *sd = side_at();
                Q4Slab b;
                b.base = codes_at();
                b.codes = word;
                b.s0 = reinterpret_cast<const uint16_t *>(sd) + (ra & 7) + g;
                b.z0 = zeros2 ? sd + Space::ZERO_AT + (ra & 15) + g : nullptr;
#pragma unroll
                for (int i = 0; i < HALVES; ++i) {
                    if (i > 0 && p_hi - panel <= 16) break;
                    b.s1 = b.s0 + 8;
                    b.z1 = b.z0 + 8;
                    q4_slab<true, SBF16, PARTS, G, Space::SCALE2_BOX, true, Space::ZERO2_BOX>(acc[i], b, xf);
                    b.base += 2048, b.s0 += 16;
                    if (zeros2) b.z0 += 16;
                }
                release();
#pragma unroll
                for (int i = 0; i < HALVES; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        if (tok[c] >= 0 && (i == 0 || p_hi - panel > 16)) {
                            float *y = sums + tok[c] * pld + row0 + 16 * i + g;
                            y[0] = fmaf(pw[c], acc[i][0][c], y[0]);
                            y[8] = fmaf(pw[c], acc[i][0][2 + c], y[8]);
                        }
                __syncwarp();
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < a.T * pld; i += MO_THREADS) {
            const int tk = pld == 16 ? i / 16 : i / MO_PANEL, r = i - tk * pld;
            float y = 0.0f;
#pragma unroll
            for (int w = 0; w < MO_WARPS; ++w) {
                y += space[w * a.T * pld + i];
                space[w * a.T * pld + i] = 0.0f;
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

template <bool BF16, bool SBF16, int G, int PARTS, bool TALL>
cudaError_t launch_one(const MoeArgs &a, const MoeMaps &m, int grid, cudaStream_t st)
{
    constexpr auto kern = moe_kernel<BF16, SBF16, G, PARTS, TALL>;
    static std::atomic<bool> configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (MO_SMEM<G, TALL>));
        if (e != cudaSuccess) return e;
        configured[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(MO_THREADS);
    cfg.dynamicSmemBytes = MO_SMEM<G, TALL>;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, m);
}

template <bool BF16, bool SBF16, int G>
cudaError_t launch_parts(const MoeArgs &a, const MoeMaps &m, int grid, cudaStream_t st)
{
    if (a.parts == 3) return launch_one<BF16, SBF16, G, 3, false>(a, m, grid, st);
    return a.tall ? launch_one<BF16, SBF16, G, 2, true>(a, m, grid, st) : launch_one<BF16, SBF16, G, 2, false>(a, m, grid, st);
}

template <bool BF16, bool SBF16>
cudaError_t launch_group(const MoeArgs &a, const MoeMaps &m, int grid, cudaStream_t st)
{
    switch (a.w1.group) {
    case 32: return launch_parts<BF16, SBF16, 32>(a, m, grid, st);
    case 64: return launch_parts<BF16, SBF16, 64>(a, m, grid, st);
    default: return launch_parts<BF16, SBF16, 128>(a, m, grid, st);
    }
}

}  // namespace

cudaError_t launch_moe(const MoeArgs &a, const MoeMaps &m, int grid, cudaStream_t st)
{
    if (a.x_bf16) return a.w1.scale_bf16 ? launch_group<true, true>(a, m, grid, st) : launch_group<true, false>(a, m, grid, st);
    return a.w1.scale_bf16 ? launch_group<false, true>(a, m, grid, st) : launch_group<false, false>(a, m, grid, st);
}

}  // namespace tc
