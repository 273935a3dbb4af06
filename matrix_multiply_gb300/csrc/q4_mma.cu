// The product of many rows of X with a 4-bit weight on the tcgen05 tensor
// cores: C = alpha X W^T + beta C, W the 128-row operand, X's rows its
// columns.
//
// W stays 4 bits up to the SM: converter warps (thread = row of W) read the
// codes that TMA brought to shared memory, widen them (q4_widen: code - zero,
// exact in X's 16-bit type) and write them to TMEM, from where
// the tensor core takes its 128-row operand; X's tiles come through shared
// memory by TMA.  Each group of k is summed from zero in one of two TMEM
// accumulators; promoting warps (thread = row of W, so a group's scale is
// one number per thread) read it and add it times the scale to fp32 sums in
// registers.  No weight is rounded, and the scales cost one packed
// multiply-add per two sums and group.  Roles, one CTA of 14 warps per SM
// (14: the register file holds 128 registers for each thread of 16 warps, 96
// for more):
//   converters   one or, for narrow tiles, two per 32 rows (each one block of
//                a pair: a narrow block's MMAs take less time than converting)
//   promoters    one or, for wide tiles, two per 32 rows (half the columns
//                each: their sums fill the registers); they write C
//   one warp for the TMA copies, one that issues the MMAs
// Few tiles: the K slices of a tile form a cluster and add their sums in
// rank order through distributed shared memory.  A short last wave: its tiles
// are cut into equal ranges of K (CUT), whose sums meet in memory; whichever
// warp comes last adds them in a fixed order.  Deterministic, all of it.
//
// What bounds it: the warps that convert.  256 k of a 128 x 128 tile take
// 1.07 us, twice the tensor core's time for it; of the ~600
// instructions per 128 k and scheduler two thirds widen codes, one warp's
// chain of them with the stores to TMEM.  Wider tiles, which would convert
// less often, have not been built: 160 columns fill TMEM with two accumulators
// and three operand stages, and their sums would need registers moved from
// other warps to the promoting ones.  The kernels of 128 and of 64 columns
// spill 44 to 52 bytes a thread.
// Measured: 4096 x 11008 x 4096 (M x N x K, bf16, groups of 128) 330 us, 1.12
// PFLOP/s, 58% of a bf16 product's measured rate, groups of 64 449, of 32 800;
// 200 x 11008 x 4096 33 us; 17 x 4096 x 4096 10 us.  The plan's figures stand
// beside its cost model.
#include "q4.cuh"

#include <atomic>

namespace tc {
namespace {

__host__ __device__ constexpr int qm_conv(int bn) { return bn > 64 ? 4 : 8; }
__host__ __device__ constexpr int qm_prom(int bn) { return bn > 64 ? 8 : 4; }
constexpr int QM_THREADS = (4 + 8 + 2) * 32;
constexpr int QM_BK = 128;                      // k of a block: the unit of every hand-over
constexpr int QM_XS = 4, QM_CS = 4;             // ring stages: X and the converted operand (a block), codes (two)
constexpr int QM_CODE_BYTES = Q4_MMA_ROWS * 128;
constexpr int QM_PART_LD = Q4_MMA_ROWS + 4;     // floats between columns of a slice's partial tile

// (never below half an SM's: a CTA holds all of TMEM, and one that waits for
// its cluster while another, on the same SM, waits for that TMEM could wait
// for ever)
__host__ __device__ constexpr int qm_smem(int bn)
{
    const int need = 1024 + QM_XS * bn * 256 + QM_CS * QM_CODE_BYTES + 512;
    return need > 120 * 1024 ? need : 120 * 1024;
}
static_assert(qm_smem(128) <= SMEM_LIMIT, "one CTA per SM");
static_assert(32 * QM_PART_LD * 4 <= QM_XS * 32 * 256 && 128 * QM_PART_LD * 4 <= QM_XS * 128 * 256,
              "a partial tile fits in the idle X ring");

// D[tmem] (+)= A[tmem] B[smem], issued by the lane whose `leader` is set.
// The whole warp runs the issuing loop, so that its addresses and
// descriptors stay in uniform registers; one lane's loop, a divergent region,
// moved every operand there for each MMA and took longer than the MMAs.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate,
                                           uint32_t leader)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void mma_commit_by(uint32_t bar, uint32_t leader)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(leader)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ unsigned ld_acquire(const unsigned *p)
{
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ unsigned atom_add_acq_rel(unsigned *p, unsigned v)
{
    unsigned old;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

// two fp32 multiply-adds, two additions
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t pack64(uint32_t lo, uint32_t hi)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}

// alpha * sum + beta * C_old of one row of W: C[off + c ldc], c < cols; the
// lanes of a warp hold neighbouring rows
template <int DT, int HB, bool BF16>
__device__ __forceinline__ void store_columns(const Q4GemmArgs &a, long long off, int cols, const uint64_t (&acc)[HB / 2])
{
    const bool whole = cols >= HB && a.beta == 0.0f;
#pragma unroll
    for (int c = 0; c < HB; ++c) {
        float v = a.alpha * q4_whole<BF16>(__uint_as_float(c & 1 ? (uint32_t)(acc[c / 2] >> 32) : (uint32_t)acc[c / 2]));
        if (!whole) {
            if (c >= cols) break;
            if (a.beta != 0.0f) v = fmaf(a.beta, load_c(a.C, off, DT), v);
        }
        store_c1(a.C, off, v, DT);
        off += a.ldc;
    }
}

struct QmUnit {
    int n0, m0, kb0, kb1, tile;
};
__device__ __forceinline__ QmUnit qm_unit(int u, int split, int tiles_m, int bn, int num_kb)
{
    const int tile = split > 1 ? u / split : u, s = u - tile * split;
    QmUnit w;
    w.tile = tile;
    w.n0 = (tile / tiles_m) * Q4_MMA_ROWS;
    w.m0 = (tile % tiles_m) * bn;
    // slices of whole pairs of blocks, as the codes are copied
    const int nb = (num_kb + 1) / 2;
    w.kb0 = split > 1 ? (int)((long long)s * nb / split) * 2 : 0;
    w.kb1 = split > 1 ? min(num_kb, (int)((long long)(s + 1) * nb / split) * 2) : num_kb;
    return w;
}

// Tiles from `whole` on are laid end to end, in pairs of blocks, and cut into
// one equal range per CTA (CUT): the pieces of this CTA's range come first,
// then the whole tiles, in turn.
struct QmCut {
    int whole, pairs, first, pieces;               // tiles taken whole; pairs of a tile; the range's tiles
    unsigned total, lo, hi;                        // pairs of all cut tiles; this CTA's range of them

    __device__ __forceinline__ unsigned bound(unsigned cta) const { return cta * total / gridDim.x; }
    // the CTA that a pair belongs to
    __device__ __forceinline__ unsigned owner(unsigned pair) const { return ((pair + 1) * gridDim.x - 1) / total; }
    __device__ __forceinline__ void init(int whole_, int tiles, int num_kb)
    {
        whole = whole_;
        pairs = (num_kb + 1) / 2;
        total = (unsigned)((tiles - whole) * pairs);
        lo = bound(blockIdx.x);
        hi = bound(blockIdx.x + 1);
        first = (int)(lo / (unsigned)pairs);
        pieces = (int)((hi - 1) / (unsigned)pairs) - first + 1;
        first += whole;
    }
    // the CTA's i-th piece
    __device__ __forceinline__ bool get(int i, int tiles_m, int bn, int num_kb, QmUnit &w) const
    {
        int tile = first + i, p0 = 0, p1 = pairs;
        if (i < pieces) {
            const unsigned t0 = (unsigned)((tile - whole) * pairs);
            p0 = (int)(max(lo, t0) - t0);
            p1 = (int)(min(hi, t0 + pairs) - t0);
        } else {
            tile = blockIdx.x + (i - pieces) * gridDim.x;
            if (tile >= whole) return false;
        }
        const int tn = (unsigned)tile / (unsigned)tiles_m;
        w = QmUnit{tn * Q4_MMA_ROWS, (tile - tn * tiles_m) * bn, 2 * p0, min(num_kb, 2 * p1), tile};
        return true;
    }
};

template <bool BF16, int BN, int G, bool CUT>
__global__ void __launch_bounds__(QM_THREADS, 1)
    q4_mma_kernel(const Q4GemmArgs a, const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmX,
                  int split, int tiles_m, int units, int whole, float *partial, unsigned *counts, unsigned *status,
                  unsigned long long timeout_ns, int debug_drop)
{
    constexpr int X_BYTES = BN * 256;              // a block of X: two halves of BN rows x 128 bytes
    constexpr int NG = QM_BK / G;                  // groups per block
    constexpr int QM_CONV = qm_conv(BN), QM_PROM = qm_prom(BN);
    constexpr int HB = BN / (QM_PROM / 4);         // columns of one promoting warp
    constexpr uint32_t TMEM_COLS = 512;
    constexpr uint32_t A_COL = 2 * BN;             // the converted operand's stages follow the accumulators
    static_assert(2 * BN + QM_XS * 64 <= 512 && BN % 32 == 0, "TMEM columns");
    constexpr uint32_t IDESC = (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) | ((uint32_t)(BN >> 3) << 17) |
                               ((uint32_t)(Q4_MMA_ROWS >> 4) << 24);
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint8_t *codes = smem + QM_XS * X_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(codes + QM_CS * QM_CODE_BYTES);
    // full: X's copies and the four converting warps of a block; empty: its MMAs
    const uint32_t full = smem_u32(bars), empty = full + 8 * QM_XS, cfull = empty + 8 * QM_XS, cempty = cfull + 8 * QM_CS,
                   dfull = cempty + 8 * QM_CS, dempty = dfull + 16, drain = dempty + 16;
    uint32_t *slot = reinterpret_cast<uint32_t *>(bars + 2 * QM_XS + 2 * QM_CS + 5);
    volatile uint32_t *abort_flag = slot + 1;

    __shared__ QmCut cut;
    const int num_kb = (int)((a.q.K + QM_BK - 1) / QM_BK);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < QM_XS; ++i) mbar_init(full + 8 * i, 5), mbar_init(empty + 8 * i, 1);
        for (int i = 0; i < QM_CS; ++i) mbar_init(cfull + 8 * i, 1), mbar_init(cempty + 8 * i, QM_CONV);
        for (int i = 0; i < 2; ++i) mbar_init(dfull + 8 * i, 1), mbar_init(dempty + 8 * i, QM_PROM);
        mbar_init(drain, 1);
        if (CUT) cut.init(whole, units, num_kb);
        *abort_flag = 0u;
        fence_barrier_init();
        prefetch_tmap(&tmC);
        prefetch_tmap(&tmX);
        griddep_launch_dependents();
    }
    __syncwarp();
    if (warp == 0) tmem_alloc(smem_u32(slot), TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    if (!CUT && split > 1) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *slot;
    griddep_wait();

    const Q4Watch watch{abort_flag, status, timeout_ns};
    const int step = split > 1 ? units : (int)gridDim.x;       // a cluster's CTAs take one unit each
    bool ok = true;
    // the CTA's pieces, one after the other
    QmUnit w;
    int u = CUT ? 0 : blockIdx.x;
    auto next = [&]() {
        if (CUT) return cut.get(u++, tiles_m, BN, num_kb, w);
        if (u >= units) return false;
        w = qm_unit(u, split, tiles_m, BN, num_kb);
        u += step;
        return true;
    };

    if (warp == QM_CONV + QM_PROM) {
        // ------------------------------------------------------ TMA copies
        if (lane == 0) {
            int xi = 0, ci = 0;                                 // copies issued
            while (ok && next()) {
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    if ((kb & 1) == 0) {
                        const int st = ci % QM_CS;
                        if (!(ok = q4_wait(cempty + 8 * st, ((ci / QM_CS) & 1) ^ 1, watch))) break;
                        mbar_arrive_expect_tx(cfull + 8 * st, QM_CODE_BYTES);
                        tma_load_2d(smem_u32(codes) + st * QM_CODE_BYTES, &tmC, cfull + 8 * st, kb * (QM_BK / 2), w.n0);
                        ++ci;
                    }
                    const int st = xi % QM_XS;
                    if (!(ok = q4_wait(empty + 8 * st, ((xi / QM_XS) & 1) ^ 1, watch))) break;
                    const bool drop = debug_drop && blockIdx.x == 0 && xi == 2;
                    mbar_arrive_expect_tx(full + 8 * st, X_BYTES + (drop ? 16 : 0));
                    tma_load_2d(smem_u32(smem) + st * X_BYTES, &tmX, full + 8 * st, kb * QM_BK, w.m0);
                    tma_load_2d(smem_u32(smem) + st * X_BYTES + X_BYTES / 2, &tmX, full + 8 * st, kb * QM_BK + 64, w.m0);
                    ++xi;
                }
            }
            // after an expired wait: the copies already issued land before shared
            // memory is released.  X's barriers may still lack the converters, so
            // the wait is for its limit.
            if (!ok) {
                for (int i = max(0, xi - QM_XS); i < xi; ++i) q4_drain(full + 8 * (i % QM_XS), (i / QM_XS) & 1);
                for (int i = max(0, ci - QM_CS); i < ci; ++i) q4_drain(cfull + 8 * (i % QM_CS), (i / QM_CS) & 1);
            }
        }
        __syncwarp();
    } else if (warp == QM_CONV + QM_PROM + 1) {
        // ------------------------------------------------------ MMA issuer
        // The warp's own latency per block paces the tensor core: each barrier
        // is looked at once ahead of time, so that a wait that is already over
        // costs nothing.
        const uint32_t leader = elect_one();
        uint32_t st = 0, ph = 0, db = 0, dph = 1;               // ring stage, accumulator, and their phases
        bool ready = false, dready = true;
        const uint64_t bd0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
        auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, q4_wait(bar, parity, watch)); };
        while (ok && next()) {
#pragma unroll 1
            for (int kb = w.kb0; kb < w.kb1; ++kb) {
                if (!ready && !(ok = wait(full + 8 * st, ph))) break;
                const uint32_t nst = (st + 1) % QM_XS, nph = st + 1 == QM_XS ? ph ^ 1u : ph;
                const uint64_t bd = bd0 + (uint64_t)(st * (X_BYTES >> 4));
                const uint32_t at = tmem + A_COL + st * 64;
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    if (!dready && !(ok = wait(dempty + 8 * db, dph))) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = i * (G / 16); k < (i + 1) * (G / 16); ++k)
                        mma_f16_ts(tmem + db * BN, at + k * 8, bd + (uint64_t)((k >> 2) * (X_BYTES >> 5) + (k & 3) * 2), IDESC,
                                   k > i * (G / 16) ? 1u : 0u, leader);
                    if (i == NG - 1) mma_commit_by(empty + 8 * st, leader);
                    mma_commit_by(dfull + 8 * db, leader);
                    db ^= 1u;
                    dph ^= db ^ 1u;
                    dready = __all_sync(0xffffffffu, mbar_test_wait(dempty + 8 * db, dph));
                }
                if (!ok) break;
                ready = __all_sync(0xffffffffu, mbar_test_wait(full + 8 * nst, nph));
                st = nst;
                ph = nph;
            }
        }
        if (!ok) {
            mma_commit_by(drain, leader);
            if (leader) q4_drain(drain, 0);
        }
        __syncwarp();
    } else if (warp < QM_CONV) {
        // ------------------------------------------------------ converters
        const int quarter = warp & 3, half = warp >> 2, row = quarter * 32 + lane;
        constexpr int BLOCKS = QM_CONV == 4 ? 2 : 1;             // blocks of a pair that a warp converts
        const int ngroups = (int)((a.q.K + G - 1) / G);
        const uint32_t to = tmem + ((uint32_t)(quarter * 32) << 16) + A_COL;
        const uint8_t *src = codes + row * 128;
        int it = 0, ci = 0;                                      // blocks and pairs before this one
        uint32_t pending = 0;                                    // the barrier of the block whose stores are under way
        auto hand_over = [&]() {
            if (!pending) return;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(pending);
            pending = 0;
        };
        while (ok && next()) {
            const uint8_t *zp = a.q.zeros ? a.q.zeros + min((long long)w.n0 + row, a.q.N - 1) : nullptr;
            // a row's zero points of a pair of blocks, loaded a pair ahead: a use
            // next to its load would wait for it
            uint8_t zn[BLOCKS][NG];
            auto load_z = [&](int kb) {
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        const int gr = (kb + (BLOCKS == 1 ? half : b)) * NG + i;
                        zn[b][i] = 8;
                        if (zp && gr < ngroups) zn[b][i] = zp[gr * a.q.lds];
                    }
            };
            load_z(w.kb0);
#pragma unroll 1
            for (int kb = w.kb0; kb < w.kb1; kb += 2, it += 2, ++ci) {
                const int cs = ci % QM_CS;
                uint32_t zz[BLOCKS][NG];
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
                    for (int i = 0; i < NG; ++i) zz[b][i] = zn[b][i] & 15u;
                if (zp) load_z(kb + 2);
                ok = __all_sync(0xffffffffu, q4_wait(cfull + 8 * cs, (ci / QM_CS) & 1, watch));
                if (!ok) break;
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b) {
                    const int bb = BLOCKS == 1 ? half : b;
                    if (kb + bb >= w.kb1) break;
                    const int as = (it + bb) % QM_XS;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {                // two halves of 64 k
                        uint32_t words[8], out[32];
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(
                                src + cs * QM_CODE_BYTES + (((4 * bb + 2 * h + v) ^ (row & 7)) << 4));
                            words[4 * v] = x.x, words[4 * v + 1] = x.y, words[4 * v + 2] = x.z, words[4 * v + 3] = x.w;
                        }
#pragma unroll
                        for (int v = 0; v < 8; ++v) {
                            uint32_t p[4];
                            q4_widen<BF16>(words[v], q4_zero_form<BF16>(zz[b][(h * 64 + v * 8) / G]), p);
#pragma unroll
                            for (int j = 0; j < 4; ++j) out[4 * v + j] = p[j];
                        }
                        if (h == 0) {
                            // the block before is handed over now: its stores have
                            // had this block's first half to complete
                            hand_over();
                            ok = __all_sync(0xffffffffu, q4_wait(empty + 8 * as, (((it + bb) / QM_XS) & 1) ^ 1, watch));
                            if (!ok) break;
                            tc_fence_after();
                        }
                        tmem_st_32x32b_x32(to + as * 64 + h * 32, out);
                    }
                    if (!ok) break;
                    pending = full + 8 * as;
                }
                if (!ok) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(cempty + 8 * cs);
            }
            it -= (w.kb1 - w.kb0) & 1;
        }
        hand_over();
    } else {
        // ------------------------------------------------------ promoting warps
        const int pw = warp - QM_CONV, quarter = pw & 3, half = pw >> 2, row = quarter * 32 + lane;
        const long long ngroups = (a.q.K + G - 1) / G;
        const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + half * HB;
        uint32_t db = 0, dph = 0;                                // accumulator and its phase
        while (ok && next()) {
            const long long n = w.n0 + row;
            uint64_t acc[HB / 2];
#pragma unroll
            for (int i = 0; i < HB / 2; ++i) acc[i] = 0ull;
            const int g0 = w.kb0 * NG, gn = (w.kb1 - w.kb0) * NG;
            // scales as they are stored, loaded two groups before their use into
            // registers that nothing touches in between (a move would wait)
            const uint16_t *sp = static_cast<const uint16_t *>(a.q.scales) + g0 * a.q.lds + (n < a.q.N ? n : 0);
            const int sn = n < a.q.N ? (int)min((long long)gn, ngroups - g0) : 0;
            uint16_t sq[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (i < sn) sq[i] = sp[i * a.q.lds];
#pragma unroll 1
            for (int i = 0; i < gn && ok; i += 2) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (i + j >= gn) break;
                    ok = __all_sync(0xffffffffu, q4_wait(dfull + 8 * db, dph, watch));
                    if (!ok) break;
                    const float s = a.q.scale_bf16 ? q4_scale_bits<true>(sq[j]) : q4_scale_bits<false>(sq[j]);
                    sq[j] = 0;
                    if (i + j + 2 < sn) sq[j] = sp[(i + j + 2) * a.q.lds];
                    tc_fence_after();
                    const uint64_t ss = pack64(__float_as_uint(s), __float_as_uint(s));
                    // 32 columns to a load: a wait is for all loads before it
#pragma unroll
                    for (int c = 0; c < HB; c += 32) {
                        uint32_t r[32];
                        if (c + 32 <= HB) {
                            tmem_ld_32x32b_x32(taddr + db * BN + c, r);
                        } else {
                            uint32_t q[16];
                            tmem_ld_x16(taddr + db * BN + c, q);
#pragma unroll
                            for (int k = 0; k < 16; ++k) r[k] = q[k];
                        }
                        tmem_ld_wait();
                        if (c + 32 >= HB) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(dempty + 8 * db);
                        }
#pragma unroll
                        for (int k = 0; k < (c + 32 <= HB ? 16 : 8); ++k)
                            acc[c / 2 + k] = fma2(ss, pack64(r[2 * k], r[2 * k + 1]), acc[c / 2 + k]);
                    }
                    db ^= 1u;
                    dph ^= db ^ 1u;
                }
            }
            if (!ok) break;
            if (!CUT && split > 1) {
                // all of the unit's MMAs have completed: the X ring is idle
                float *part = reinterpret_cast<float *>(smem);
#pragma unroll
                for (int c = 0; c < HB; ++c)
                    part[(half * HB + c) * QM_PART_LD + row] =
                        __uint_as_float(c & 1 ? (uint32_t)(acc[c / 2] >> 32) : (uint32_t)acc[c / 2]);
                continue;
            }
            bool last = true;
            if (CUT && w.kb1 - w.kb0 != num_kb) {
                // A piece of the tile: the sums go to this CTA's place for its
                // first or its last piece, and whichever warp finds all the
                // others written adds them up; no warp waits for another.  Of two
                // pieces the later warp adds the earlier's to its own; more are
                // added in order of k.
                const unsigned t0 = (unsigned)((w.tile - whole) * cut.pairs);
                const unsigned c0 = cut.owner(t0), c1 = cut.owner(t0 + cut.pairs - 1);
                unsigned *count = counts + (w.tile - whole) * QM_PROM + pw;
                // this warp's part of a place: four columns at a time, a lane's next to each other
                const auto place = [&](unsigned cta, bool second) {
                    return reinterpret_cast<float4 *>(partial) + (size_t)(2 * cta + second) * (BN * Q4_MMA_ROWS / 4) +
                           pw * (HB * 8) + lane;
                };
                unsigned before = 0;
                if (c1 == c0 + 1) {
                    if (lane == 0) before = ld_acquire(count);
                    before = __shfl_sync(0xffffffffu, before, 0);
                }
                if (before == 0) {
                    float4 *mine = place(blockIdx.x, w.tile != cut.first);
#pragma unroll
                    for (int c = 0; c < HB / 4; ++c)
                        __stcg(mine + 32 * c, make_float4(__uint_as_float((uint32_t)acc[2 * c]),
                                                          __uint_as_float((uint32_t)(acc[2 * c] >> 32)),
                                                          __uint_as_float((uint32_t)acc[2 * c + 1]),
                                                          __uint_as_float((uint32_t)(acc[2 * c + 1] >> 32))));
                    __syncwarp();
                    if (lane == 0) before = atom_add_acq_rel(count, 1u);
                    before = __shfl_sync(0xffffffffu, before, 0);
                }
                last = before == c1 - c0;
                if (last) {
                    // lane 0 alone has acquired the others' sums; the shuffle
                    // that passed its count on orders no memory
                    __syncwarp();
                    if (lane == 0) *count = 0u;                // as the next launch expects it
                    if (c1 > c0 + 1)
#pragma unroll
                        for (int c = 0; c < HB / 2; ++c) acc[c] = 0ull;
#pragma unroll 1
                    for (unsigned q = c0; q <= c1; ++q) {
                        if (c1 == c0 + 1 && q == blockIdx.x) continue;
                        // the first owner's piece may be its last one; the others' are their first
                        const float4 *p = place(q, cut.bound(q) < t0);
#pragma unroll
                        for (int c = 0; c < HB / 4; ++c) {
                            const float4 v = __ldcg(p + 32 * c);
                            acc[2 * c] = add2(acc[2 * c], pack64(__float_as_uint(v.x), __float_as_uint(v.y)));
                            acc[2 * c + 1] = add2(acc[2 * c + 1], pack64(__float_as_uint(v.z), __float_as_uint(v.w)));
                        }
                    }
                }
            }
            if (last && n < a.q.N) {
                const int cols = min(HB, a.M - w.m0 - half * HB);
                const long long off = (long long)(w.m0 + half * HB) * a.ldc + n;
                if (a.c_dtype == TC_F32)
                    store_columns<TC_F32, HB, BF16>(a, off, cols, acc);
                else
                    store_columns<BF16 ? TC_BF16 : TC_F16, HB, BF16>(a, off, cols, acc);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (!CUT && split > 1) {
        cluster_sync();              // every slice's partial tile is in its CTA's shared memory
        w = qm_unit(blockIdx.x, split, tiles_m, BN, num_kb);
        const int rank = (int)cluster_ctarank();
        const int c0 = rank * BN / split, c1 = (rank + 1) * BN / split;
        const uint32_t base = smem_u32(smem);
        for (int i = c0 * Q4_MMA_ROWS + threadIdx.x; i < c1 * Q4_MMA_ROWS; i += QM_THREADS) {
            const int c = i / Q4_MMA_ROWS, r = i % Q4_MMA_ROWS;
            const long long n = w.n0 + r;
            if (n >= a.q.N || w.m0 + c >= a.M || *abort_flag) continue;
            const uint32_t o = base + (uint32_t)(c * QM_PART_LD + r) * 4u;
            float p[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < split) p[q] = ld_shared_cluster_f32(mapa_shared(o, (uint32_t)q));
            float v = p[0];
#pragma unroll
            for (int q = 1; q < 8; ++q)
                if (q < split) v += p[q];
            v = q4_whole<BF16>(v) * a.alpha;
            const long long off = (long long)(w.m0 + c) * a.ldc + n;
            if (a.beta != 0.0f) v = fmaf(a.beta, load_c(a.C, off, a.c_dtype), v);
            store_c1(a.C, off, v, a.c_dtype);
        }
        __syncwarp();
        cluster_sync();              // no CTA releases its shared memory while a peer may read it
    }
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
}

template <bool BF16, int BN, int G, bool CUT = false>
cudaError_t launch_one(const Q4GemmArgs &a, const Q4MmaPlan &p, cudaStream_t st)
{
    constexpr auto kern = q4_mma_kernel<BF16, BN, G, CUT>;
    constexpr int smem = qm_smem(BN);
    static std::atomic<bool> configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        configured[dev].store(true, std::memory_order_release);
    }
    return launch_dependent(kern, dim3((unsigned)p.grid), dim3(QM_THREADS), smem, st, (unsigned)p.split, a, p.codes, p.x,
                            p.split, p.tiles_m, p.tiles_n * p.tiles_m * p.split, p.whole, p.partial, p.counts, p.status,
                            p.timeout_ns, p.debug_drop);
}

template <bool BF16, int BN>
cudaError_t launch_group(const Q4GemmArgs &a, const Q4MmaPlan &p, cudaStream_t st)
{
    if constexpr (BN == 128)
        if (p.whole < p.tiles_n * p.tiles_m) switch (a.q.group) {
            case 32: return launch_one<BF16, BN, 32, true>(a, p, st);
            case 64: return launch_one<BF16, BN, 64, true>(a, p, st);
            default: return launch_one<BF16, BN, 128, true>(a, p, st);
            }
    switch (a.q.group) {
    case 32: return launch_one<BF16, BN, 32>(a, p, st);
    case 64: return launch_one<BF16, BN, 64>(a, p, st);
    default: return launch_one<BF16, BN, 128>(a, p, st);
    }
}

}  // namespace

int q4_mma_max_clusters(int split)
{
    // (every instantiation fills an SM: one stands for all)
    constexpr auto kern = q4_mma_kernel<true, 128, 128, false>;
    constexpr int smem = qm_smem(128);
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)split);
    cfg.blockDim = dim3(QM_THREADS);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) return 0;
    return n;
}

cudaError_t launch_q4_mma(const Q4GemmArgs &a, const Q4MmaPlan &p, cudaStream_t st)
{
    if (p.split < 1 || p.split > 8 || p.grid < 1 || p.grid % p.split != 0 ||
        (p.split > 1 && p.grid != p.tiles_n * p.tiles_m * p.split))
        return cudaErrorInvalidValue;
    const long long cut = (long long)(p.tiles_n * p.tiles_m - p.whole) * ((a.q.K + 255) / 256);
    if (cut > 0 && (p.bn != 128 || p.split > 1 || cut < p.grid || cut * p.grid > 0xffffffffll || !p.partial || !p.counts))
        return cudaErrorInvalidValue;
    switch (p.bn) {
    case 32: return a.x_bf16 ? launch_group<true, 32>(a, p, st) : launch_group<false, 32>(a, p, st);
    case 64: return a.x_bf16 ? launch_group<true, 64>(a, p, st) : launch_group<false, 64>(a, p, st);
    case 96: return a.x_bf16 ? launch_group<true, 96>(a, p, st) : launch_group<false, 96>(a, p, st);
    case 128: return a.x_bf16 ? launch_group<true, 128>(a, p, st) : launch_group<false, 128>(a, p, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace tc
