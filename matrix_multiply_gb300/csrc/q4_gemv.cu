// The product of at most 16 rows of X with a 4-bit weight: C = alpha X W^T +
// beta C.  Every code is read once, so HBM bounds it; the kernel is built
// around that stream.
//   * A persistent CTA per SM owns a range of W's rows, equal to one row
//     between CTAs, cut into blocks of at most 16 rows, or 32 (MT 2).  Its 16
//     warps divide K: a warp takes the same 256 k (a slab) of every block, so
//     its share of X stays in registers for the whole kernel.  When K has at
//     most 8 slabs, several groups of warps take different blocks; when it has
//     more than 16, a warp has several slabs and reads its share of X once per
//     six blocks of 16 rows (three, for more than 8 rows of X).
//   * Each warp streams its slabs through a ring of its own in shared
//     memory, filled by TMA (codes, scales, zero points of a block's slab),
//     several pieces ahead; nothing is shared with other warps until, every
//     few blocks, the warps' sums of those blocks are added in a fixed order.
//   * When N leaves fewer than 16 rows to a CTA, K above 4096 is split over a
//     cluster of CTAs, whose sums are added in rank order through distributed
//     shared memory.
//   * The multiply-adds run on mma.sync m16n8k16 with W as the 16-row
//     operand (see q4_slab).
// Fixed orders everywhere: the result is deterministic.
//
// Measured (M x N x K, X and C in 16 bits but where said), with the share of
// a plain copy's rate that the bytes come to:
//   1 x 4096 x 4096, groups of 128              4.3 us   30%
//   4 x 4096 x 11008, of 64 with zero points    8.8 us   42%
//   16 x 11008 x 4096, of 32, C in fp32        12.4 us   32%
// An empty launch takes 3.1; after it the kernel is bound by the issue and the
// latencies of the widening and its bookkeeping (per 16 rows x 256 k 420
// instructions in all at the second of these, 590 at the third; schedulers
// issue in 45% of the cycles, 16 warps being what the registers hold), not by
// HBM.  mma.sync
// rather than tcgen05: with at most 16 columns the tensor cores are idle
// either way, and W goes from the ring to the operand's registers without a
// second pass through shared memory or TMEM.
#include "q4.cuh"

#include <atomic>

namespace tc {
namespace {

constexpr int GV_WARPS = 16;
// A stage of a warp's ring: codes, scales, zero points of a block of MT
// operands of 16 rows
template <int MT>
struct GvStage {
    static constexpr int STAGES = MT == 1 ? 3 : 2;
    static constexpr int SCALE_BOX = 8 + 16 * MT, ZERO_BOX = 16 + 16 * MT;
    static constexpr int SCALE_AT = 2048 * MT, ZERO_AT = SCALE_AT + 8 * 2 * SCALE_BOX;
    static constexpr int BYTES = MT == 1 ? 3072 : 5120;        // a multiple of the swizzle's 1024
    static_assert(ZERO_AT % 128 == 0 && ZERO_AT + 8 * ZERO_BOX <= BYTES && BYTES % 1024 == 0, "stage layout");
};
static_assert(GvStage<1>::SCALE_BOX == Q4_SCALE_BOX && GvStage<1>::ZERO_BOX == Q4_ZERO_BOX, "boxes");
template <int MT>
constexpr int GV_RING = GV_WARPS * GvStage<MT>::STAGES * GvStage<MT>::BYTES;
constexpr int GV_TILE_LD = 20;             // floats between X rows of a 16-row partial tile: conflict-free both ways

// blocks whose partial tiles are held before they are added up
template <int NT, int MT>
__host__ __device__ constexpr int gv_hold() { return (NT == 1 ? 6 : 3) / MT; }
template <int NT>
__host__ __device__ constexpr int gv_tile() { return NT * 8 * GV_TILE_LD; }       // floats
template <int NT, int MT>
__host__ __device__ constexpr int gv_smem()
{
    return 1024 + GV_RING<MT> + (GV_WARPS + 1) * gv_hold<NT, MT>() * MT * gv_tile<NT>() * 4 +
           GV_WARPS * GvStage<MT>::STAGES * 8;
}
static_assert(gv_smem<1, 1>() <= SMEM_LIMIT && gv_smem<2, 1>() <= SMEM_LIMIT && gv_smem<1, 2>() <= SMEM_LIMIT,
              "one CTA per SM");

template <bool BF16, bool SBF16, int NT, int G, int MT>
__global__ void __launch_bounds__(GV_WARPS * 32, 1)
    q4_gemv_kernel(const Q4GemmArgs a, const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmT,
                   const __grid_constant__ CUtensorMap tmS, const __grid_constant__ CUtensorMap tmZ, int ksplit, int rows,
                   int nblk, int block_rows, int tail_rows, unsigned *status, unsigned long long timeout_ns, int debug_drop)
{
    constexpr int GP = Q4_SLAB / G;                // groups per slab
    constexpr int TILE = gv_tile<NT>();
    constexpr int HOLD = gv_hold<NT, MT>();
    using Stage = GvStage<MT>;
    constexpr int S = Stage::STAGES;
    extern __shared__ uint8_t raw[];
    uint8_t *ring = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    float *tiles = reinterpret_cast<float *>(ring + GV_RING<MT>);      // [HOLD * MT][GV_WARPS][TILE]
    float *sums = tiles + GV_WARPS * HOLD * MT * TILE;                 // [HOLD * MT][TILE], for the cluster
    uint64_t *bars = reinterpret_cast<uint64_t *>(sums + HOLD * MT * TILE);

    const int warp = uniform_warp(), lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int K = (int)a.q.K;
    const int nslab = (K - 1) / Q4_SLAB + 1;
    int cluster = blockIdx.x, rank = 0, s_lo = 0, s_hi = nslab;
    if (ksplit > 1) {
        cluster = blockIdx.x / (unsigned)ksplit;
        rank = blockIdx.x - cluster * ksplit;
        s_lo = (unsigned)(rank * nslab) / (unsigned)ksplit;
        s_hi = (unsigned)((rank + 1) * nslab) / (unsigned)ksplit;
    }
    const int mine = s_hi - s_lo;                                      // slabs of this CTA (at least 1)
    int wk_n = GV_WARPS, wr_n = 1, wr = 0, wk = warp;                  // warps along K, groups along the blocks
    if (mine < GV_WARPS) {
        wk_n = mine;
        wr_n = ksplit > 1 ? 1u : (unsigned)GV_WARPS / (unsigned)mine;
        wr = (unsigned)warp / (unsigned)mine;
        wk = warp - wr * mine;
    }
    const bool active = wr < wr_n;
    // slabs of this warp in every block: one, unless the CTA's part of K is above 4096
    const int per = !active ? 0 : mine <= GV_WARPS ? 1 : (mine - wk + GV_WARPS - 1) / GV_WARPS;
    const long long r_lo = (long long)cluster * rows;
    const int nrows = (int)min((long long)rows, a.q.N - r_lo);

    const uint32_t my_ring = smem_u32(ring) + warp * (S * Stage::BYTES);
    const uint32_t my_bar = smem_u32(bars + warp * S);
    const bool zeros = a.q.zeros != nullptr;
    if (lane == 0) {
        prefetch_tmap(&tmC);
        prefetch_tmap(&tmS);
        if (zeros) prefetch_tmap(&tmZ);
        for (int i = 0; i < S; ++i) mbar_init(my_bar + 8 * i, 1);
        fence_barrier_init();
    }
    __syncwarp();
    griddep_launch_dependents();
    griddep_wait();

    // the warp's pieces, fetched in order
    const uint32_t leader = elect_one();
    uint32_t beside = GP * (2 * Stage::SCALE_BOX + (zeros ? Stage::ZERO_BOX : 0));
    if (debug_drop && blockIdx.x == 0) beside += 16;
    // blocks with rows in them
    const int have = nrows == rows ? nblk : (int)((unsigned)(nrows - 1) / (unsigned)block_rows) + 1;
    int f_first = wr, f_h = 0, f_s = 0, fetched = 0;
    uint32_t f_at = 0;                             // the stage's offset in the ring
    // the order of the pieces: HOLD blocks at a time, of these slab by slab
    auto fetch = [&]() {                           // the whole warp
        if (f_first >= have || per == 0) return;
        const int blk = f_first + f_h * wr_n, row = (int)r_lo + blk * block_rows, slab = s_lo + wk + f_s * GV_WARPS;
        const uint32_t st = my_ring + f_at, bar = my_bar + f_at / (Stage::BYTES / 8);
        const bool tail = MT > 1 && blk == nblk - 1;
        arrive_expect_by(bar, (tail ? tail_rows : block_rows) * 128 + beside, leader);
        tma_load_2d_by(st, tail ? &tmT : &tmC, bar, slab * (Q4_SLAB / 2), row, leader);
        tma_load_2d_by(st + Stage::SCALE_AT, &tmS, bar, row & ~7, slab * GP, leader);
        if (zeros) tma_load_2d_by(st + Stage::ZERO_AT, &tmZ, bar, row & ~15, slab * GP, leader);
        ++fetched;
        f_at = f_at == (S - 1) * Stage::BYTES ? 0u : f_at + Stage::BYTES;
        if (++f_h == HOLD || f_first + f_h * wr_n >= have) {
            f_h = 0;
            if (++f_s == per) f_s = 0, f_first += HOLD * wr_n;
        }
    };
#pragma unroll 1
    for (int i = 0; i < S; ++i) fetch();

    // this warp's share of X: of one slab, for the whole kernel, or of the
    // slab at hand
    const uint16_t *X = static_cast<const uint16_t *>(a.X);
    const bool x_vec = (reinterpret_cast<uintptr_t>(X) & 15u) == 0 && (a.ldx & 7) == 0;
    uint32_t xf[NT][8][4];
    auto load_xf = [&](int slab) {
        const bool whole = x_vec && slab < K / Q4_SLAB;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 8; ++j) xf[nt][j][0] = xf[nt][j][1] = xf[nt][j][2] = xf[nt][j][3] = 0u;
            if (nt * 8 + g < a.M)
                q4_load_slab(xf[nt], X + (nt * 8 + g) * a.ldx, (long long)slab * Q4_SLAB + t * 8, K, whole);
        }
    };
    if (per > 0) load_xf(s_lo + wk);
    const uint32_t word = q4_first_word(g, t);

    // outputs of X row `col`, W rows r and r + 1 of a block
    auto write_out = [&](int blk, int col, int r, float v0, float v1) {
        const int left = min(block_rows, nrows - blk * block_rows) - r;
        if (left <= 0 || col >= a.M) return;
        const long long off = col * a.ldc + r_lo + blk * block_rows + r;
        v0 = q4_whole<BF16>(v0) * a.alpha, v1 = q4_whole<BF16>(v1) * a.alpha;
        if (a.beta != 0.0f) {
            v0 = fmaf(a.beta, load_c(a.C, off, a.c_dtype), v0);
            if (left > 1) v1 = fmaf(a.beta, load_c(a.C, off + 1, a.c_dtype), v1);
        }
        store_c1(a.C, off, v0, a.c_dtype);
        if (left > 1) store_c1(a.C, off + 1, v1, a.c_dtype);
    };

    const Q4Watch watch{nullptr, status, timeout_ns};
    int stage = 0, parity = 0;
    bool ok = true;
    // phases of HOLD blocks per group of warps
    for (int first = ksplit > 1 ? 0 : wr; first < nblk; first += HOLD * wr_n) {
        if (!active) {
            if (ksplit == 1) break;
        }
        int held = 0;
        if (active) held = wr_n == 1 ? min(HOLD, have - first) : min(HOLD, (have - first + wr_n - 1) / wr_n);
        for (int s = 0; s < per; ++s) {
            if (per > 1) load_xf(s_lo + wk + s * GV_WARPS);
            for (int h = 0; h < held; ++h) {
                const int blk = first + h * wr_n, row = (int)(r_lo & 15) + blk * block_rows;   // (only its low bits are used)
                const bool second = MT > 1 && nrows - blk * block_rows > 16;
                float acc[MT][NT][4];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) acc[m][nt][0] = acc[m][nt][1] = acc[m][nt][2] = acc[m][nt][3] = 0.0f;
                ok = ok && q4_wait(my_bar + 8 * stage, parity, watch);
                __syncwarp();
                const uint8_t *st = ring + (warp * S + stage) * Stage::BYTES;
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if (m > 0 && !second) break;
                    Q4Slab b;
                    b.base = st + 2048 * m;
                    b.codes = word;
                    b.s0 = reinterpret_cast<const uint16_t *>(st + Stage::SCALE_AT) + (row & 7) + g + 16 * m;
                    b.s1 = b.s0 + 8;
                    b.z0 = zeros ? st + Stage::ZERO_AT + (row & 15) + g + 16 * m : nullptr;
                    b.z1 = b.z0 + 8;
                    q4_slab<BF16, SBF16, NT, G, Stage::SCALE_BOX, false, Stage::ZERO_BOX>(acc[m], b, xf);
                }
                __syncwarp();                                          // every lane has read the piece
                if (__all_sync(0xffffffffu, ok)) fetch();
                if (++stage == S) stage = 0, parity ^= 1;
                // the block's partial tiles, a slab at a time
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if (m > 0 && !second) break;
                    float *tile = tiles + ((h * MT + m) * GV_WARPS + warp) * TILE + 2 * t * GV_TILE_LD + g;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float *p = tile + (nt * 8 + (e & 1)) * GV_TILE_LD + 8 * (e >> 1);
                            if (s > 0) acc[m][nt][e] += *p;
                            *p = acc[m][nt][e];
                        }
                }
            }
        }
        __syncwarp();
        if (active) {
            q4_group_sync(wr, wk_n);
            // a pair of threads per four rows of one X row: each adds every
            // other warp's tile, in warp order, then the two join
            const int half = lane & 1;
            for (int e = (wk * 32 + lane) >> 1; e < HOLD * MT * NT * 32; e += wk_n * 16) {
                const int hm = e / (NT * 32), h = hm / MT, c = (e >> 2) % (NT * 8), r = (e & 3) * 4;
                const int o = c * GV_TILE_LD + r, blk = first + h * wr_n, r0 = hm % MT * 16;
                const bool in = h < held && c < a.M && nrows - blk * block_rows > r0;
                const float *p = tiles + (hm * GV_WARPS + warp - wk) * TILE + o;
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < GV_WARPS; w += 2)
                    if (in && w + half < wk_n) {
                        const float4 x = *reinterpret_cast<const float4 *>(p + (w + half) * TILE);
                        v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
                    }
                v.x += __shfl_xor_sync(0xffffffffu, v.x, 1);
                v.y += __shfl_xor_sync(0xffffffffu, v.y, 1);
                v.z += __shfl_xor_sync(0xffffffffu, v.z, 1);
                v.w += __shfl_xor_sync(0xffffffffu, v.w, 1);
                if (!in) continue;
                if (ksplit == 1)
                    write_out(blk, c, r0 + r + 2 * half, half ? v.z : v.x, half ? v.w : v.y);
                else if (!half)
                    *reinterpret_cast<float4 *>(sums + hm * TILE + o) = v;
            }
        }
        if (ksplit > 1) {
            __syncwarp();
            cluster_sync();
            const uint32_t base = smem_u32(sums);
            const int count = min(HOLD, nblk - first);
            // the phase's outputs, pairs of rows, dealt out to the ranks' threads
            for (int i = rank * (GV_WARPS * 32) + threadIdx.x; i < count * MT * NT * 64; i += ksplit * GV_WARPS * 32) {
                const int hm = i / (NT * 64), h = hm / MT, c = (i >> 3) % (NT * 8), r = (i & 7) * 2, r0 = hm % MT * 16;
                if (c >= a.M || nrows - (first + h) * block_rows <= r0) continue;
                const uint32_t o = base + (uint32_t)(hm * TILE + c * GV_TILE_LD + r) * 4u;
                float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q < ksplit) {
                        const uint32_t peer = mapa_shared(o, (uint32_t)q);
                        v0 += ld_shared_cluster_f32(peer);
                        v1 += ld_shared_cluster_f32(peer + 4);
                    }
                write_out(first + h, c, r0 + r, v0, v1);
            }
            __syncwarp();
            cluster_sync();      // the sums are read before they are overwritten, or their CTA ends
        } else if (first + HOLD * wr_n < nblk) {
            q4_group_sync(wr, wk_n);      // the tiles are read before the next phase's are written
        }
    }
    // after an expired wait: copies still in flight land (within a limit)
    // before shared memory is released
    if (!ok && lane == 0)
        for (int i = 0; i < S; ++i) {
            const int n = (fetched + S - 1 - i) / S;                   // copies into this stage
            if (n > 0) q4_drain(my_bar + 8 * i, (uint32_t)(n - 1) & 1u);
        }
}

template <bool BF16, bool SBF16, int NT, int G, int MT>
cudaError_t launch_one(const Q4GemmArgs &a, const Q4GemvPlan &p, cudaStream_t st)
{
    constexpr auto kern = q4_gemv_kernel<BF16, SBF16, NT, G, MT>;
    constexpr int smem = gv_smem<NT, MT>();
    static std::atomic<bool> configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        configured[dev].store(true, std::memory_order_release);
    }
    return launch_dependent(kern, dim3((unsigned)(p.clusters * p.ksplit)), dim3(GV_WARPS * 32), smem, st,
                            (unsigned)p.ksplit, a, p.codes, p.tail, p.scales, p.zeros, p.ksplit, p.rows, p.nblk,
                            p.block_rows, p.tail_rows, p.status, p.timeout_ns, p.debug_drop);
}

template <bool BF16, bool SBF16, int NT, int G>
cudaError_t launch_tall(const Q4GemmArgs &a, const Q4GemvPlan &p, cudaStream_t st)
{
    if constexpr (NT == 1)
        if (p.tall == 2) return launch_one<BF16, SBF16, NT, G, 2>(a, p, st);
    return launch_one<BF16, SBF16, NT, G, 1>(a, p, st);
}

template <bool BF16, bool SBF16, int NT>
cudaError_t launch_group(const Q4GemmArgs &a, const Q4GemvPlan &p, cudaStream_t st)
{
    switch (a.q.group) {
    case 32: return launch_tall<BF16, SBF16, NT, 32>(a, p, st);
    case 64: return launch_tall<BF16, SBF16, NT, 64>(a, p, st);
    default: return launch_tall<BF16, SBF16, NT, 128>(a, p, st);
    }
}

}  // namespace

int q4_gemv_max_clusters(int ksplit)
{
    // split ranges are short: blocks of 16 rows; the larger instantiation's
    // shared memory
    if (ksplit == 1) {
        int dev = 0, sms = 0;
        cudaGetDevice(&dev);
        return cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? sms : 0;
    }
    constexpr auto kern = q4_gemv_kernel<true, true, 2, 128, 1>;
    constexpr int smem = gv_smem<2, 1>();
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ksplit);
    cfg.blockDim = dim3(GV_WARPS * 32);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ksplit;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) return 0;
    return n;
}

cudaError_t launch_q4_gemv(const Q4GemmArgs &a, const Q4GemvPlan &p, cudaStream_t st)
{
    if (a.M < 1 || a.M > Q4_GEMV_MAX_ROWS || p.ksplit < 1 || p.ksplit > 8 || p.clusters < 1 || p.tall < 1 || p.tall > 2 ||
        (p.tall > 1 && (p.ksplit > 1 || a.M > 8)) || p.block_rows < 1 || p.block_rows > 16 * p.tall || p.tail_rows < 1 ||
        p.tail_rows > p.block_rows)
        return cudaErrorInvalidValue;
    const bool wide = a.M > 8;
    if (a.x_bf16)
        return a.q.scale_bf16 ? (wide ? launch_group<true, true, 2>(a, p, st) : launch_group<true, true, 1>(a, p, st))
                              : (wide ? launch_group<true, false, 2>(a, p, st) : launch_group<true, false, 1>(a, p, st));
    return a.q.scale_bf16 ? (wide ? launch_group<false, true, 2>(a, p, st) : launch_group<false, true, 1>(a, p, st))
                          : (wide ? launch_group<false, false, 2>(a, p, st) : launch_group<false, false, 1>(a, p, st));
}

}  // namespace tc
