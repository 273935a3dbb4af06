// Launch descriptions shared by the host API (api.cpp) and the kernels.
// Plain structs; no PyTorch types anywhere in the library.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>
#include <utility>

namespace tc {

// Launch `kern` as a programmatic dependent of the stream's previous kernel
// (clusters of `cluster` CTAs when above 1).  Its CTAs may be scheduled as
// soon as every CTA of that kernel has executed
// griddepcontrol.launch_dependents or exited, so the launch and the
// kernel's set-up overlap the previous kernel's last CTAs; every kernel
// launched this way runs griddepcontrol.wait -- which returns once the
// previous grid has completed and its memory operations are visible --
// before its first global memory access.  Behind anything but a kernel
// (a copy, an event, another stream's work) the launch is ordered as usual.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                             unsigned cluster, Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// Tile geometry of the tensor-core kernel.  Every output tile is BM rows by
// BN columns; the K loop steps BK elements (one 128-byte swizzle row of a
// 16-bit type) per pipeline stage.
constexpr int BM = 128;
constexpr int BK = 64;
constexpr int MMA_K = 16;                       // K of one kind::f16 tcgen05.mma
constexpr int MMA_THREADS = 192;                // 4 epilogue warps, TMA warp, MMA warp (plain GEMM kernels)
constexpr int SMEM_LIMIT = 232448;              // max dynamic shared memory per block
constexpr int EPI_STAGE_BYTES = 4096;           // one 32 x 32 output chunk (fp32 worst case)

// Epilogue warps: four (warp w reads TMEM lanes 32w..32w+31), or, for the
// fused bias/activation epilogue and for grouped launches (`epi` true),
// eight -- two per TMEM lane quarter, each taking every other 32-column
// chunk -- so that CUDA-core epilogue work takes half as long: the tail
// tile's, which no next tile hides, and the plain-store epilogue of ragged
// problems, which otherwise holds the accumulator longer than the next
// tile's K loop runs.  The one-CTA 192-wide tile keeps four (its fifth
// pipeline stage needs the space).
__host__ __device__ constexpr int epi_warps(int bn, int cg, bool epi) { return (epi && !(bn == 192 && cg == 1)) ? 8 : 4; }
__host__ __device__ constexpr int mma_threads(int bn, int cg, bool epi) { return (epi_warps(bn, cg, epi) + 2) * 32; }
// Epilogue staging per warp: with four warps two chunk buffers (one TMA
// store may still be reading the other), except for the 192-wide tiles,
// which keep one buffer so that one more pipeline stage fits (the one-CTA
// tile's 40 KB stages: a fifth; the pair's 28 KB: a seventh; their K loops
// are bound by the latency the ring covers and their shapes run a single
// wave, which drains once); with eight warps one buffer each.  The plain-store
// path's 32 x 32-float transpose buffer is one such buffer, so a warp's
// staging never overlaps another warp's (a launch may use both paths: C by
// plain stores, split-K partial tiles by TMA stores).  Buffers start at
// multiples of 1024 bytes, the alignment the swizzled TMA layouts assume
// (the swizzle uses the absolute shared address).
__host__ __device__ constexpr int epi_bufs(int bn, int cg, bool epi)
{
    return (epi_warps(bn, cg, epi) == 8 || bn == 192) ? 1 : 2;
}
__host__ __device__ constexpr int epi_warp_bytes(int bn, int cg, bool epi)
{
    return epi_warps(bn, cg, epi) == 8 ? EPI_STAGE_BYTES : epi_bufs(bn, cg, epi) == 1 ? 5120 : 8192;
}
__host__ __device__ constexpr int epi_smem(int bn, int cg, bool epi) { return epi_warps(bn, cg, epi) * epi_warp_bytes(bn, cg, epi); }

__host__ __device__ constexpr int smem_reserve(int bn, int cg, bool epi)   // alignment slack + barriers + epilogue staging
{
    return 1024 + 256 + epi_smem(bn, cg, epi);
}

// One pipeline stage of a CTA: its 128 rows of A and its share of B (all BN
// columns for a single CTA; BN/2 for each CTA of a pair running
// tcgen05.mma.cta_group::2 on a 256 x BN tile).
__host__ __device__ constexpr int stage_bytes(int bn, int cg) { return (BM + bn / cg) * BK * 2; }
__host__ __device__ constexpr int tmem_cols(int bn)
{
    return (2 * bn <= 128) ? 128 : (2 * bn <= 256) ? 256 : 512;
}
__host__ __device__ constexpr int mma_stages(int bn, int cg, bool epi = false)
{
    return ((SMEM_LIMIT - smem_reserve(bn, cg, epi)) / stage_bytes(bn, cg)) > 8
               ? 8
               : ((SMEM_LIMIT - smem_reserve(bn, cg, epi)) / stage_bytes(bn, cg));
}
__host__ __device__ constexpr int mma_smem_bytes(int bn, int cg, bool epi = false)
{
    return mma_stages(bn, cg, epi) * stage_bytes(bn, cg) + smem_reserve(bn, cg, epi);
}

// Device-side arguments of the tensor-core kernel (the two TMA descriptors
// travel as separate __grid_constant__ parameters).
struct MmaArgs {
    int M, N, K;
    int num_kb;            // ceil(K / BK)
    int tiles_m, tiles_n;  // per batch entry
    int tiles_per_batch;
    int batch;
    // Work units: output tiles in the linear (band-swizzled) order, each cut
    // into K slices.  Tiles [0, seg0_tiles) have seg0_split slices each, the
    // remaining tiles seg1_split slices each; unit u enumerates (tile, slice)
    // pairs in that order.  A tile with more than one slice parks its
    // partial sums in ws slot (u - split_base) and the last slice to finish
    // reduces them in slice order.
    int seg0_tiles, seg0_split, seg1_split;
    int split_base;
    int total_units;
    int group_m;           // rasterisation band height, in tile rows
    int a_kmajor, b_kmajor;
    int a_3d, b_3d;        // 3-D descriptors: the batch index is the third coordinate
    // MN-major operand read through a chunked 3-D descriptor (64 elements,
    // K rows, 64-element chunks): one copy brings a CTA's whole share of
    // the operand for a K block instead of one copy per 64-wide chunk
    int a_chunked, b_chunked;
    uint32_t idesc;        // tcgen05 instruction descriptor
    float alpha, beta;
    void *C;
    long long ldc, stride_c;
    int c_dtype;           // TC_F16 / TC_BF16 / TC_F32
    int c_vec_ok;          // 16-byte vector loads/stores allowed on C
    int c_tma;             // C is written by TMA stores through the third descriptor
    int c_3d;              // that descriptor is 3-D (batch index third)
    float *ws;             // split-K partial tiles (written through the fourth descriptor)
    unsigned *status;      // device status word (0 = fine)
    unsigned long long timeout_ns;
    int debug_drop_tfull;  // test hook: never signal the first tile's accumulator
    // fused epilogue: bias (N values of c_dtype, or null) and activation
    // (TC_ACT_*) applied after alpha/beta, before the one rounding; a
    // per-column scale (N floats, or null) applied to the accumulator before
    // alpha/beta (the int8 path's dequantisation)
    const void *bias;
    int act;
    const float *col_scale;
    int slice_kb;          // on-chip int8 accumulation: K blocks per exact slice
    // one-CTA tiles over fewer than BM rows of a K-major A: its copies carry
    // only the rows that exist (rounded up to 8) and a stage this many fewer
    // bytes; the tile's other rows hold stale data, which reaches only
    // output rows beyond M (never stored)
    int a_short_bytes;
};

struct MmaLaunch {
    int bn;
    int cg;      // CTAs per tile: 1, or 2 for a CTA pair (cluster of two)
    int i8acc;   // int8 slices summed in TMEM (BN = 128 only; args.slice_kb, col_scale)
    // split-K inside one launch: the args.seg0_split K slices of a tile form
    // one cluster and add their partial tiles through distributed shared
    // memory (BN 64 or 128, one CTA per unit: grid == args.total_units)
    int csplit;
    int grid;    // CTAs (a multiple of cg)
    CUtensorMap tmA, tmB, tmC, tmW;   // A, B, C and the split-K workspace
    MmaArgs args;
};

cudaError_t launch_mma(const MmaLaunch &L, cudaStream_t st);

// A group of independent problems in one persistent launch.  Every problem
// has its own TMA descriptors and epilogue fields; all share the kernel
// shape (BN, CTAs per tile) and take one K slice per tile.  Unit u (one
// output tile) belongs to the problem p with unit_begin[p] <= u <
// unit_begin[p + 1]; the table travels as a kernel parameter.
constexpr int GROUP_MAX = 64;
struct GroupInfo {
    int M, N, num_kb;
    int tiles_m, tiles_n;
    int unit_begin;
    int a_kmajor, b_kmajor;
    uint32_t idesc;
    int c_dtype, c_vec_ok, c_tma;
    float alpha, beta;
    void *C;
    long long ldc;
};
struct GroupTable {
    CUtensorMap tmA[GROUP_MAX], tmB[GROUP_MAX], tmC[GROUP_MAX];
    GroupInfo info[GROUP_MAX];
    int count;
};
// L.args carries the launch-wide fields (total_units, group_m, status,
// timeout); the per-problem ones come from the table.
cudaError_t launch_mma_grouped(const MmaLaunch &L, const GroupTable &g, cudaStream_t st);
// Largest number of CTA pairs of the BN-wide pair kernel that can be
// resident at once on the current device (0 if the pair kernel cannot run).
int max_active_pairs(int bn);
// Largest number of S-CTA clusters of the BN-wide cluster-split kernel
// resident at once on the current device (0 if such a cluster cannot run).
int max_active_csplit_clusters(int bn, int S);

// Split-K reduction: tiles [first_tile, first_tile + ntiles) each have S
// fp32 partial tiles (rows_per_tile x bn, row-major) at
// ws + ((tile - first_tile) * S + s) * rows_per_tile * bn.
struct ReduceArgs {
    const float *ws;
    int rows_per_tile, bn;
    int first_tile, ntiles, S;
    int tiles_m, tiles_n, tiles_per_batch, group_m;
    int M, N;
    float alpha, beta;
    void *C;
    long long ldc, stride_c;
    int c_dtype, c_vec_ok;
    const void *bias;      // fused epilogue, as in MmaArgs
    int act;
    const float *col_scale;
    int int_sum;           // the slices are integers: add them as 64-bit integers
    // a status word in device memory (or null): nonzero when one of the
    // GEMM's bounded waits expired, so some partial tiles were never
    // written; the reduction then leaves C alone
    const unsigned *status;
};
// One CTA of bn threads per 8 (or, for small reductions, 4) rows of a tile,
// 8 (4) columns per thread; c_vec_ok allows 16-byte accesses to C.
cudaError_t launch_reduce(const ReduceArgs &r, cudaStream_t st);

// Static scratch of the entry point that allocates nothing: split-K partial
// tiles (at most NOALLOC_PARTIAL_BYTES) and one status word.
constexpr size_t NOALLOC_PARTIAL_BYTES = size_t(16) << 20;
constexpr size_t NOALLOC_SCRATCH_BYTES = NOALLOC_PARTIAL_BYTES + 256;
struct NoallocScratch {
    float *partials;
    unsigned *status;
};
// Device addresses of the static scratch on the current device (looked up
// once per device).
cudaError_t noalloc_scratch(NoallocScratch *out);

// Skinny products (gemv.cu): Out = alpha * (X W^T) (* scale[w row]) +
// beta * Out_old for X with at most GEMV_MAX_ROWS rows.  X is [rows_x, K]
// (f16 or bf16, row stride ldx elements), W is [rows_w, K] (X's type, or
// int8 when w_i8; row stride ldw elements); the output element of (X row
// i, W row j) is at C + i * c_sx + j * c_sw (elements of c_dtype).  The
// cluster kernel splits K across a cluster of ksplit CTAs (1, 2, 4 or 8)
// whose sums are added in rank order.
constexpr int GEMV_MAX_ROWS = 16;
struct GemvArgs {
    const void *X, *W;
    void *C;
    const float *scale;    // per W row, or null
    int rows_x, rows_w;
    long long K, ldx, ldw;
    long long c_sx, c_sw;
    int c_dtype;
    float alpha, beta;
    int x_vec, w_vec;      // 16-byte loads allowed: 16-byte aligned base and row stride
    int w_i8, x_bf16;
    int ksplit;
    // row-range kernel (16-byte aligned rows of X and W): `grid` persistent
    // CTAs (at most rows_w), CTA c owning W rows [c rows_w / grid,
    // (c + 1) rows_w / grid) -- or, with block_rows, whole 16-row blocks
    // [16 (c nb / grid), 16 ((c + 1) nb / grid)) of the nb = ceil(rows_w / 16)
    // blocks; ksplit is then unused
    int rowrange, grid, block_rows;
};
cudaError_t launch_gemv(const GemvArgs &a, cudaStream_t st);
// fp32 FFMA kernel (exact fp32, ascending-k fused multiply-add chain)
struct FfmaArgs {
    int M, N, K;
    int batch;
    int ta, tb;
    const float *A, *B;
    float *C;
    long long lda, ldb, ldc;
    long long stride_a, stride_b, stride_c;
    float alpha, beta;
};
enum FfmaTile { FFMA_SMALL = 0, FFMA_LARGE = 1, FFMA_PANEL = 2 };
cudaError_t launch_ffma(const FfmaArgs &a, int tile, cudaStream_t st);

// Relaxed fp32: a stored fp32 matrix (rows x cols, leading dimension ld_src)
// becomes three bf16 copies placed side by side along its K dimension (the
// columns when k_along_cols, else the rows), part j = hi or lo per
// parts[j] (0 = hi = bf16(x), 1 = lo = bf16(x - hi)), in a buffer with
// leading dimension ld_dst (a multiple of 64) and a 256-byte aligned base.
struct SplitArgs {
    const float *src;
    uint16_t *dst;
    long long rows, cols, ld_src, ld_dst;
    int k_along_cols;
    int parts[3];
};
cudaError_t launch_split(const SplitArgs &a, cudaStream_t st);

// int8 matrix (rows x cols, leading dimension ld_src) -> bf16, or f16 when
// to_f16 (both exact for int8), with leading dimension ld_dst (a multiple
// of 64) and a 256-byte aligned base.
struct WidenArgs {
    const int8_t *src;
    uint16_t *dst;
    long long rows, cols, ld_src, ld_dst;
    int to_f16;
};
cudaError_t launch_widen(const WidenArgs &a, cudaStream_t st);

// Copy a strided batch of 16-bit matrices (rows x cols, leading dimension
// ld_src) into a buffer with leading dimension ld_dst (a multiple of 64) and
// a 256-byte aligned base, so that TMA can read it.
struct PackArgs {
    const uint16_t *src;
    uint16_t *dst;
    long long rows, cols, ld_src, ld_dst, stride_src, stride_dst;
    int batch;
};
// Up to PACK_MAX such copies in one launch (block_begin is filled in by
// launch_pack: the first CTA of each copy, then the total).
constexpr int PACK_MAX = 128;
struct PackBatch {
    int count;
    long long block_begin[PACK_MAX + 1];
    PackArgs seg[PACK_MAX];
};
cudaError_t launch_pack(PackBatch &pb, cudaStream_t st);

// ------------------------------------------------------------- 4-bit weights
// A tc_q4_weight after validation (the public header states the format):
// row n's codes at codes + n * ldw / 2 bytes, the scale of (n, k) at
// scales[(k / group) * lds + n], the zero point beside it (8 when null).
struct Q4View {
    const uint8_t *codes;
    const void *scales;
    const uint8_t *zeros;
    long long N, K, ldw, lds;
    int group, scale_bf16;
};

// Quantising and reading back: chunks of at least 1024 k, one per grid row.
constexpr int Q4_MATRIX_MAX_K = 65535 * 1024;
struct Q4QuantArgs {
    const void *W;
    long long ld;
    int w_dtype;
    Q4View q;              // codes, scales and zeros are written
};
cudaError_t launch_q4_quantize(const Q4QuantArgs &a, cudaStream_t st);
struct Q4DequantArgs {
    Q4View q;
    void *V;
    long long ld;
    int v_dtype;
};
cudaError_t launch_q4_dequantize(const Q4DequantArgs &a, cudaStream_t st);

// C[M, N] = alpha * X[M, K] W^T + beta * C
struct Q4GemmArgs {
    Q4View q;
    const void *X;
    void *C;
    int M, x_bf16, c_dtype;
    long long ldx, ldc;
    float alpha, beta;
};

// For at most Q4_GEMV_MAX_ROWS rows of X, streaming W (q4_gemv.cu).
// The grid is `clusters` clusters of ksplit CTAs; cluster c owns the rows
// [c * rows, (c + 1) * rows) of W, in nblk blocks of block_rows <= 16 tall rows
// (tall 1 or 2; the last of a tall 2 range has tail_rows),
// and its CTA of rank r the slabs [r n / ksplit, (r + 1) n / ksplit) of the
// n = ceil(K / 256) slabs of 256 k.
constexpr int Q4_GEMV_MAX_ROWS = 16;
struct Q4GemvPlan {
    int clusters, ksplit, rows, nblk, block_rows, tall, tail_rows;
    CUtensorMap codes, tail, scales, zeros;
    unsigned *status;
    unsigned long long timeout_ns;
    int debug_drop;            // test hook: the first CTA's copies never complete
};
// boxes of the maps: {128 bytes, block_rows (tail_rows)} with the 128-byte
// swizzle, {8 + 16 tall scales, 256 / group}, {16 + 16 tall zeros, 256 / group}
constexpr int Q4_SCALE_BOX = 24, Q4_ZERO_BOX = 32;
cudaError_t launch_q4_gemv(const Q4GemmArgs &a, const Q4GemvPlan &p, cudaStream_t st);
// clusters of ksplit CTAs of that kernel resident at once (0: none)
int q4_gemv_max_clusters(int ksplit);

// The same for more rows of X, on the tcgen05 tensor cores (q4_mma.cu): tiles
// of 128 rows of W by bn rows of X, bn in {32, 64, 96, 128}; with split > 1
// the K slices of a tile form a cluster whose sums are added on chip (one
// unit per CTA); with bn 128 the last tiles can be cut instead.  X is readable
// by TMA (16-byte base and row pitch).
constexpr int Q4_MMA_ROWS = 128;
constexpr int Q4_MMA_COUNTS = 8;      // promoting warps of a tile
struct Q4MmaPlan {
    int bn, split, tiles_n, tiles_m, grid;
    int whole;                 // tiles taken whole; the rest is cut into one equal range per CTA (split 1)
    float *partial;            // 2 grid tiles of fp32, where whole < tiles
    unsigned *counts;          // Q4_MMA_COUNTS per tile that is cut, 0 before and after a launch
    CUtensorMap codes, x;      // boxes {128 bytes, 128 rows} and {64 elements, bn rows}, 128-byte swizzle
    unsigned *status;
    unsigned long long timeout_ns;
    int debug_drop;            // test hook: the first CTA's third copy of X never completes
};
cudaError_t launch_q4_mma(const Q4GemmArgs &a, const Q4MmaPlan &p, cudaStream_t st);
// clusters of `split` CTAs of that kernel resident at once (0: none)
int q4_mma_max_clusters(int split);

// The mixture-of-experts layer (the public header states the formulas): one
// cooperative launch of `grid` CTAs (moe.cu).
struct MoeArgs {
    int T, H, I, E, k;
    int x_bf16, r_dtype, y_dtype, renorm;
    int parts;             // bf16 parts of h: 2 or 3
    int tall;              // pieces of two units or 32 rows (parts 2; rows of inter 16-byte multiples)
    int rows8, panel;      // stage 2: a CTA's rows of hidden / 8, and those of a panel (8 .. 32)
    const void *X, *R;
    void *Y;
    long long ldx, ldr, ldy;
    Q4View w1, w2;         // the same group and scale type
    int *ids;              // [T, k] or null
    float *p;              // [T, k] or null
    float *logits;         // scratch [T, E]
    uint16_t *h;           // scratch, bf16: h's leading parts, each [T k, ldh]
    long long ldh;         // I rounded up to 8
    unsigned *sync;        // the grid barrier's word, 0 before the first launch of this grid size that uses it
    unsigned *status;
    unsigned long long timeout_ns;
    int debug_drop;        // test hook: 1 the second CTA misses the first grid barrier, 2 the first CTA's copies never complete
};
// gate_up is seen as [2 experts][inter rows][..]: one copy brings 8 rows of
// gate and the same 8 of up.  Boxes: codes {128 bytes, 8 rows, 2} with the
// 128-byte swizzle, scales {16, 256 / group, 2} where rows of inter are 16-byte
// multiples (s1_3d; else {16, 256 / group}, two copies), zero points {32, ..}
// likewise.  down, with r = 16 rows or, tall, 32: codes {128 bytes, the least
// of r and panel}, scales {8 + r, 256 / group}, zero points {16 + r, 256 / group}.
constexpr int MOE_SCALE_BOX = 16;
// tokens up to which a tall panel of stage 2 can have 32 rows (else 16)
constexpr int moe_panel_tokens(int group) { return group == 32 ? 24 : 32; }
struct MoeMaps {
    CUtensorMap c1, s1, z1, c2, s2, z2;
    int s1_3d, z1_3d;
};
cudaError_t launch_moe(const MoeArgs &a, const MoeMaps &m, int grid, cudaStream_t st);

}  // namespace tc
