// The product of at most 16 rows of X with a 4-bit weight: C = alpha X W^T +
// beta C.  Every code is read once, so HBM bounds it; the kernel is built
// around that stream.
//   * A persistent CTA per SM owns a range of W's rows, equal to one row
//     between CTAs, cut into blocks of at most 16 rows.  Its 16 warps divide
//     K: a warp takes the same 256 k (a slab) of every block, so its share of
//     X stays in registers for the whole kernel.  When K has fewer than 9
//     slabs, several groups of warps take different blocks.
//   * Each warp streams its slabs through a ring of its own in shared
//     memory, filled by TMA (codes, scales, zero points of a block's slab),
//     several pieces ahead; nothing is shared with other warps until their
//     sums of a block are added in warp order.
//   * K above 4096 is split over a cluster of CTAs, whose sums are added in
//     rank order through distributed shared memory.
//   * The multiply-adds run on mma.sync m16n8k16 with W as the 16-row
//     operand (see q4_slab).
// Fixed orders everywhere: the result is deterministic.
#include "q4.cuh"

#include <atomic>

namespace tc {
namespace {

constexpr int GV_WARPS = 16;
constexpr int GV_STAGES = 3;
constexpr int GV_STAGE_BYTES = 3072;       // codes 2048, scales <= 384, zero points <= 256 (512-byte aligned stages)
constexpr int GV_SCALE_AT = 2048, GV_ZERO_AT = 2560;
constexpr int GV_TILE_LD = 20;             // floats between X rows of a 16-row partial tile: conflict-free both ways
constexpr int GV_SUM_BLOCKS = 16;          // blocks whose sums a cluster member holds between two exchanges
constexpr int GV_RING = GV_WARPS * GV_STAGES * GV_STAGE_BYTES;

template <int NT>
__host__ __device__ constexpr int gv_tile() { return NT * 8 * GV_TILE_LD; }       // floats
template <int NT>
__host__ __device__ constexpr int gv_smem()
{
    return 512 + GV_RING + (2 * GV_WARPS + GV_SUM_BLOCKS) * gv_tile<NT>() * 4 + GV_WARPS * GV_STAGES * 8;
}

__device__ __forceinline__ void bar_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

template <bool BF16, int NT, int G>
__global__ void __launch_bounds__(GV_WARPS * 32, 1)
    q4_gemv_kernel(const Q4GemmArgs a, const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmS,
                   const __grid_constant__ CUtensorMap tmZ, int ksplit, int rows, int nblk, int block_rows,
                   unsigned *status, unsigned long long timeout_ns)
{
    constexpr int GP = Q4_SLAB / G;                // groups per slab
    constexpr int TILE = gv_tile<NT>();
    constexpr int COLS = NT * 8;
    extern __shared__ uint8_t raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 511) & ~static_cast<uintptr_t>(511));
    float *red = reinterpret_cast<float *>(ring + GV_RING);            // [2][GV_WARPS][TILE]
    float *sums = red + 2 * GV_WARPS * TILE;                           // [GV_SUM_BLOCKS][TILE]
    uint64_t *bars = reinterpret_cast<uint64_t *>(sums + GV_SUM_BLOCKS * TILE);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int cluster = blockIdx.x / ksplit, rank = blockIdx.x - cluster * ksplit;
    const int nslab = (int)((a.q.K + Q4_SLAB - 1) / Q4_SLAB);
    const int s_lo = (int)((long long)rank * nslab / ksplit), s_hi = (int)((long long)(rank + 1) * nslab / ksplit);
    const int mine = s_hi - s_lo;                                      // slabs of this CTA (at least 1)
    const int wk_n = min(mine, GV_WARPS), wr_n = GV_WARPS / wk_n;      // warps along K, groups along the blocks
    const int wr = warp / wk_n, wk = warp - wr * wk_n;
    const bool active = wr < wr_n;
    const int per = active ? (mine - wk + wk_n - 1) / wk_n : 0;        // slabs of this warp in every block
    const long long r_lo = (long long)cluster * rows, r_hi = min(a.q.N, r_lo + rows);
    const int nb = active ? (nblk - wr + wr_n - 1) / wr_n : 0;         // blocks of this warp's group: wr, wr + wr_n, ..
    const int items = nb * per;

    const uint32_t my_ring = smem_u32(ring) + warp * (GV_STAGES * GV_STAGE_BYTES);
    const uint32_t my_bar = smem_u32(bars + warp * GV_STAGES);
    if (lane == 0) {
        for (int i = 0; i < GV_STAGES; ++i) mbar_init(my_bar + 8 * i, 1);
        fence_barrier_init();
        prefetch_tmap(&tmC);
        prefetch_tmap(&tmS);
    }
    __syncwarp();
    griddep_launch_dependents();
    griddep_wait();

    const bool zeros = a.q.zeros != nullptr;
    const uint32_t bytes = 2 * block_rows * 64 + GP * (Q4_SCALE_BOX * 2 + (zeros ? Q4_ZERO_BOX : 0));
    int i_blk = wr, i_s = 0, i_stage = 0;                              // the next item to fetch
    auto fetch = [&]() {
        const int row = (int)(r_lo + (long long)i_blk * block_rows);
        const int slab = s_lo + wk + i_s * wk_n;
        const uint32_t st = my_ring + i_stage * GV_STAGE_BYTES, bar = my_bar + 8 * i_stage;
        mbar_arrive_expect_tx(bar, bytes);
        tma_load_2d(st, &tmC, bar, slab * (Q4_SLAB / 2), row);
        tma_load_2d(st + Q4_HALF_BYTES, &tmC, bar, slab * (Q4_SLAB / 2) + 64, row);
        tma_load_2d(st + GV_SCALE_AT, &tmS, bar, row & ~7, slab * GP);
        if (zeros) tma_load_2d(st + GV_ZERO_AT, &tmZ, bar, row & ~15, slab * GP);
        if (++i_stage == GV_STAGES) i_stage = 0;
        if (++i_s == per) i_s = 0, i_blk += wr_n;
    };
    int fetched = min(items, GV_STAGES);                               // lane 0's count
    if (lane == 0)
        for (int i = 0; i < fetched; ++i) fetch();
    __syncwarp();

    // this warp's share of X: of one slab, for the whole kernel; with several
    // slabs a warp (K above 4096 * 8) it is read again for each piece
    const uint16_t *X = static_cast<const uint16_t *>(a.X);
    const bool x_vec = (reinterpret_cast<uintptr_t>(X) & 15u) == 0 && (a.ldx & 7) == 0;
    uint32_t xf[NT][8][4];
    auto load_xf = [&](int slab) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (nt * 8 + g < a.M)
                    v = q4_load_x(X + (nt * 8 + g) * a.ldx, (long long)slab * Q4_SLAB + j * 32 + t * 8, a.q.K, x_vec);
                xf[nt][j][0] = v.x, xf[nt][j][1] = v.y, xf[nt][j][2] = v.z, xf[nt][j][3] = v.w;
            }
    };
    if (per > 0) load_xf(s_lo + wk);

    auto write_out = [&](int blk, int e, float v) {
        const int col = e >> 4, r = e & 15;
        const long long n = r_lo + (long long)blk * block_rows + r;
        if (r < block_rows && n < r_hi && col < a.M) {
            const long long off = col * a.ldc + n;
            v *= a.alpha;
            store_c1(a.C, off, a.beta != 0.0f ? fmaf(a.beta, load_c(a.C, off, a.c_dtype), v) : v, a.c_dtype);
        }
    };

    int stage = 0, parity = 0, buf = 0;
    bool ok = true;
    // phases of GV_SUM_BLOCKS blocks when a cluster exchanges its sums, else one
    const int phase_blocks = ksplit > 1 ? GV_SUM_BLOCKS : nblk;
    int blk = wr;
    for (int first = 0; first < nblk; first += phase_blocks) {
        const int last = min(nblk, first + phase_blocks);
        for (; active && blk < last; blk += wr_n) {
            float acc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
            const int row = (int)(r_lo + (long long)blk * block_rows);
            for (int s = 0; s < per; ++s) {
                if (per > 1) load_xf(s_lo + wk + s * wk_n);
                ok = ok && q4_wait(my_bar + 8 * stage, parity, status, timeout_ns);
                __syncwarp();
                const uint32_t st = my_ring + stage * GV_STAGE_BYTES;
                Q4Slab b;
                b.codes = st + g * 64 + t * 4;
                b.s0 = st + GV_SCALE_AT + ((row & 7) + g) * 2;
                b.s1 = b.s0 + 16;
                b.ss = Q4_SCALE_BOX * 2;
                b.z0 = zeros ? st + GV_ZERO_AT + (row & 15) + g : 0u;
                b.z1 = b.z0 + 8;
                b.zs = Q4_ZERO_BOX;
                q4_slab<BF16, NT, G>(acc, b, xf, g, a.q.scale_bf16);
                __syncwarp();
                if (fetched < items && lane == 0 && ok) fetch(), ++fetched;
                if (++stage == GV_STAGES) stage = 0, parity ^= 1;
            }
            // the group's warps add their tiles in warp order; two buffers, so
            // that one barrier a block is enough
            float *tile = red + (buf * GV_WARPS + warp) * TILE;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    tile[(nt * 8 + 2 * t + (e & 1)) * GV_TILE_LD + g + 8 * (e >> 1)] = acc[nt][e];
            bar_sync(wr, wk_n * 32);
            const float *tiles = red + (buf * GV_WARPS + wr * wk_n) * TILE;
            for (int e = wk * 32 + lane; e < COLS * 16; e += wk_n * 32) {
                const int at = (e >> 4) * GV_TILE_LD + (e & 15);
                float v = tiles[at];
                for (int w = 1; w < wk_n; ++w) v += tiles[w * TILE + at];
                if (ksplit == 1)
                    write_out(blk, e, v);
                else
                    sums[(blk - first) * TILE + at] = v;
            }
            buf ^= 1;
        }
        if (ksplit > 1) {
            __syncwarp();
            cluster_sync();
            const uint32_t base = smem_u32(sums);
            for (int i = threadIdx.x; i < (last - first) * COLS * 16; i += GV_WARPS * 32) {
                const int b = i / (COLS * 16), e = i - b * (COLS * 16);
                if (b % ksplit != rank) continue;
                const uint32_t at = base + (uint32_t)(b * TILE + (e >> 4) * GV_TILE_LD + (e & 15)) * 4u;
                float part[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q < ksplit) part[q] = ld_shared_cluster_f32(mapa_shared(at, (uint32_t)q));
                float v = part[0];
#pragma unroll
                for (int q = 1; q < 8; ++q)
                    if (q < ksplit) v += part[q];
                write_out(first + b, e, v);
            }
            __syncwarp();
            cluster_sync();      // the sums are read before they are overwritten, or their CTA ends
        }
    }
    // after an expired wait: copies still in flight land (within a limit)
    // before shared memory is released
    if (!ok && lane == 0)
        for (int i = 0; i < GV_STAGES; ++i) {
            const int n = (fetched + GV_STAGES - 1 - i) / GV_STAGES;   // copies into this stage
            const uint64_t t0 = globaltimer_ns();
            while (n > 0 && !mbar_try_wait(my_bar + 8 * i, (uint32_t)(n - 1) & 1u) && globaltimer_ns() - t0 < 200000000ull) {}
        }
}

template <bool BF16, int NT, int G>
cudaError_t launch_one(const Q4GemmArgs &a, const Q4GemvPlan &p, cudaStream_t st)
{
    constexpr auto kern = q4_gemv_kernel<BF16, NT, G>;
    constexpr int smem = gv_smem<NT>();
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
                            (unsigned)p.ksplit, a, p.codes, p.scales, p.zeros, p.ksplit, p.rows, p.nblk, p.block_rows,
                            p.status, p.timeout_ns);
}

}  // namespace

int q4_gemv_max_clusters(int ksplit)
{
    // the largest instantiation's shared memory; the others need no more
    if (ksplit == 1) {
        int dev = 0, sms = 0;
        cudaGetDevice(&dev);
        return cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? sms : 0;
    }
    constexpr auto kern = q4_gemv_kernel<true, 2, 128>;
    constexpr int smem = gv_smem<2>();
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
    if (a.M < 1 || a.M > Q4_GEMV_MAX_ROWS || p.ksplit < 1 || p.ksplit > 8 || p.clusters < 1 || p.block_rows < 1 ||
        p.block_rows > 16)
        return cudaErrorInvalidValue;
    const int g = a.q.group == 32 ? 0 : a.q.group == 64 ? 1 : 2;
    switch ((a.x_bf16 ? 6 : 0) + (a.M > 8 ? 3 : 0) + g) {
    case 0: return launch_one<false, 1, 32>(a, p, st);
    case 1: return launch_one<false, 1, 64>(a, p, st);
    case 2: return launch_one<false, 1, 128>(a, p, st);
    case 3: return launch_one<false, 2, 32>(a, p, st);
    case 4: return launch_one<false, 2, 64>(a, p, st);
    case 5: return launch_one<false, 2, 128>(a, p, st);
    case 6: return launch_one<true, 1, 32>(a, p, st);
    case 7: return launch_one<true, 1, 64>(a, p, st);
    case 8: return launch_one<true, 1, 128>(a, p, st);
    case 9: return launch_one<true, 2, 32>(a, p, st);
    case 10: return launch_one<true, 2, 64>(a, p, st);
    default: return launch_one<true, 2, 128>(a, p, st);
    }
}

}  // namespace tc
