// Products of 8-bit matrices (e4m3 with a scale for each block of 128, see
// glu_quant.cuh) on the fifth-generation tensor cores of sm_103a, dense and by
// expert, plain or with the gated activation and the quantisation of its result
// in the epilogue:
//
//     P_w[m, n] = sum_b sa[m, b] sw[n / 128, b] sum_{k in block b} a[m, k] w[n, k]
//     glu_gemm_q_nt    d = round(P_b)
//     glu_gemm_q_fwd   y, y_scale = quantised act(P_gate) * P_up
//
// tcgen05.mma kind::f8f6f4 sums the 128 products of one block (fp32, in tensor
// memory); the epilogue warps read that block's sums with tcgen05.ld and add
// them, times sa * sw, to fp32 sums in registers, while the tensor cores work
// on the next block in the other half of tensor memory.  So scales need not be
// powers of two: sa * sw is rounded once to fp32 (it loses bits below 2^-126) and
// each block's sum once, and no sum over more than 128 terms is left to the
// tensor core.
//
// Two kernels:
//   * wide: a pair of blocks (cta_group::2) per tile of 256 rows of a; one
//     thread holds half of one row's columns (128 sums), so the row scale is one
//     float per thread and a row's largest magnitude needs two threads;
//   * narrow, for few rows: the weights take the 128 lanes of the MMA and the
//     rows of a its N (16 to 64), so no tensor-core row is wasted on absent
//     rows and the time is the weights' trip from HBM; long sums over few tiles
//     are split over the blocks of a cluster, which add their parts in a fixed
//     order through distributed shared memory.
// By expert, a tile belongs to one expert: tiles are counted from the offsets
// on the device, so the host needs to know only the total number of rows.
//
// Every wait is bounded as in glu_gemm.cu: one that runs out is counted for
// glu_wait_timeouts and leaves the block's remaining outputs unwritten.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "glu.h"
#include "glu_kernels.cuh"
#include "glu_internal.h"
#include "glu_quant.cuh"
#include "glu_tensor.cuh"

namespace glu {
namespace gemmq {

using namespace glu::gemm;

constexpr int BM = 128;             // tensor-memory lanes
constexpr int BK = 128;             // K per stage = one scale block = one 128-byte swizzle row
constexpr int kMaxGroups = 1024;
constexpr int kBox = 32;            // outputs leave through boxes of 32 rows of 64 bytes

struct Params {
    const float *sa;                // row scales
    int64_t sa_stride;              // floats
    const float *sw0, *sw1;         // weight scales: b; or gate and up
    int64_t sw_stride, sw_group;    // floats: per 128 rows, per expert
    char *y;
    int64_t y_stride;               // bytes
    float *ys;                      // gated: y's scales
    int64_t ys_stride;              // floats
    const int32_t *offsets;         // by expert: n_groups + 1 row offsets, else NULL
    int n_groups;                   // 1 without offsets
    int M, N;                       // rows of a in all, output columns
    int k_tiles;
    int n_blocks;                   // column tiles
    int group_m;                    // wide: row tiles side by side in the tile order
    int m_tiles;                    // row tiles; with offsets the most there can be
    int tma_store;                  // wide: y's base, rows and width are 16-byte multiples: it leaves through the copy engine
};

static __device__ unsigned int g_q_timeouts;

// Instruction descriptor of kind::f8f6f4: fp32 accumulator (bits 4-5 = 1), A
// and B e4m3 (format 0), both K-major, N >> 3 at bits 17-22, M >> 4 at 24-28.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N)
{
    return (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

template <int CTAS>
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    if constexpr (CTAS == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}

// A box of a 3-D tensor (column, row, expert) into this block's shared memory.
template <int CTAS>
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    if constexpr (CTAS == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
            "[%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
            "{%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
}

// The same box of the first expert into L2 only.
__device__ __forceinline__ void prefetch3(const CUtensorMap *map, int x, int y)
{
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(0)
                 : "memory");
}

// 16 consecutive fp32 columns of this warp's 32 tensor-memory lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Arrives on a barrier of the pair after tensor-memory reads, which the
// tcgen05 fence before it orders.  The barrier orders nothing else, so the
// arrival is a release at block scope only: at cluster scope each one waited
// for the warp's whole memory traffic (1262 us instead of 581 at 4096 x 4096 x
// 2 x 14336).
__device__ __forceinline__ void arrive_pair(uint32_t bar_cluster)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// wait_parity that asks once before it reads the clock: the waits of the K loop
// are handshakes of a few hundred cycles, one after the other.
__device__ __forceinline__ bool wait_quick(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done || wait_parity(bar, parity);
}

// Waits for this thread's tensor-memory loads; the registers pass through, so
// that no use of them can be moved before the wait.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])::"memory");
}

// One lane of a converged warp.  The MMA warp runs its loop as a whole and only
// issues from one lane: the loop's values stay warp-uniform, which is how the
// MMAs take them.
__device__ __forceinline__ bool elect_one()
{
    uint32_t yes;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(yes));
    return yes != 0;
}

__device__ __forceinline__ float ld_shared(uint32_t addr)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float ld_cluster(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ f2 pair(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }

// act(g) * u with the activation at its fp32-accurate degree (the forward's
// shorter series would show in y's scale, a float).
template <class Act>
__device__ __forceinline__ f2 gated(f2 g, f2 u)
{
    f2 a, d;
    Act::bwd2(g, &a, &d);
    return mul2(a, u);
}

// gated() of two pairs.  The sigmoid forms take one reciprocal for all four,
// 1 / (1 + e) of each from that of their product (in [1, 16]): the special
// functions, eight cycles a warp each, are what a gated tile's end waits for.
// The minimum drops a NaN (e is at most 1 otherwise), which would reach the
// other three through the product; the factor g keeps it in its own column
// (0.7 % of the time at 4096 x 4096 x 2 x 14336; a branch for NaN took 3.7 %).
template <class Act>
__device__ __forceinline__ void gated4(f2 &g0, f2 u0, f2 &g1, f2 u1)
{
    if constexpr (std::is_same<Act, Silu>::value || std::is_same<Act, GeluTanh>::value) {
        f2 w0 = g0, w1 = g1;
        if constexpr (std::is_same<Act, GeluTanh>::value) {
            w0 = GeluTanh::arg2(g0);
            w1 = GeluTanh::arg2(g1);
        }
        f2 e0 = exp2_twice(mul2(abs2(w0), splat(kNegHalfLog2e)));
        f2 e1 = exp2_twice(mul2(abs2(w1), splat(kNegHalfLog2e)));
        e0 = make_float2(fminf(e0.x, 1.0f), fminf(e0.y, 1.0f));
        e1 = make_float2(fminf(e1.x, 1.0f), fminf(e1.y, 1.0f));
        const f2 d0 = add2(e0, splat(1.0f)), d1 = add2(e1, splat(1.0f));
        const float p0 = d0.x * d0.y, p1 = d1.x * d1.y;
        const float r = rcp_ftz(p0 * p1), r0 = r * p1, r1 = r * p0;
        const f2 m0 = make_float2(w0.x >= 0.0f ? 1.0f : e0.x, w0.y >= 0.0f ? 1.0f : e0.y);
        const f2 m1 = make_float2(w1.x >= 0.0f ? 1.0f : e1.x, w1.y >= 0.0f ? 1.0f : e1.y);
        g0 = mul2(mul2(g0, mul2(m0, mul2(splat(r0), make_float2(d0.y, d0.x)))), u0);
        g1 = mul2(mul2(g1, mul2(m1, mul2(splat(r1), make_float2(d1.y, d1.x)))), u1);
    } else {
        g0 = gated<Act>(g0, u0);
        g1 = gated<Act>(g1, u1);
    }
}

// ---------------------------------------------------------------- tiles

// First and last row of group e, clamped to the matrix and to each other, so
// that no offset can lead out of it.
__device__ __forceinline__ void group_rows(const Params &p, int e, int &lo, int &hi)
{
    lo = 0;
    hi = p.M;
    if (p.offsets) {
        lo = min(max(p.offsets[e], 0), p.M);
        hi = min(max(p.offsets[e + 1], lo), p.M);
    }
}

// prefix[e] = row tiles of the groups before e, for e <= n_groups; called by
// every thread of the block, followed by a barrier.  Sums stop at m_tiles,
// which offsets that do not decrease never pass: with others the tiles are
// wrong but inside every matrix.
__device__ __forceinline__ void count_tiles(const Params &p, int rows_per_tile, int *prefix)
{
    if (!p.offsets) {
        if (threadIdx.x == 0) {
            prefix[0] = 0;
            prefix[1] = p.m_tiles;
        }
        return;
    }
    if (threadIdx.x >= 32) return;
    // each lane counts a run of neighbouring groups (their offsets come in one
    // trip to memory), then the lanes' sums are scanned
    const int lane = threadIdx.x, per = (p.n_groups + 31) / 32, first = lane * per;
    int sum = 0;
#pragma unroll 8
    for (int i = 0; i < per; ++i) {
        const int e = first + i;
        if (e < p.n_groups) {
            int lo, hi;
            group_rows(p, e, lo, hi);
            sum = min(sum + min((hi - lo + rows_per_tile - 1) / rows_per_tile, p.m_tiles), p.m_tiles);
            prefix[e + 1] = sum;
        }
    }
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int w = __shfl_up_sync(0xFFFFFFFFu, before, o);
        if (lane >= o) before = min(before + w, p.m_tiles);
    }
    before = __shfl_up_sync(0xFFFFFFFFu, before, 1);
    if (lane == 0) before = prefix[0] = 0;
    for (int e = first; e < min(first + per, p.n_groups); ++e) prefix[e + 1] = min(prefix[e + 1] + before, p.m_tiles);
}

struct Tile {
    int e;          // expert
    int row, end;   // first row of the tile, end of the expert's rows
    int nb;         // column tile
};

// Tile t: the experts one after the other, each with its row tiles side by side
// (group_m at a time) along the column tiles, so that neighbouring tiles share
// a weight slice.
__device__ __forceinline__ Tile tile_at(const Params &p, const int *prefix, int t, int rows_per_tile)
{
    Tile r;
    const int q = t / p.n_blocks;
    int a = 0, b = p.n_groups;
    while (b - a > 1) {                 // prefix[a] <= q < prefix[b]
        const int m = (a + b) >> 1;
        if (prefix[m] <= q)
            a = m;
        else
            b = m;
    }
    r.e = a;
    const int blocks = prefix[a + 1] - prefix[a];
    const int local = t - prefix[a] * p.n_blocks;
    const int per = p.group_m * p.n_blocks;
    const int first = (local / per) * p.group_m;
    const int side = min(blocks - first, p.group_m);
    const int in = local % per;
    group_rows(p, a, r.row, r.end);
    r.row += (first + in % side) * rows_per_tile;
    r.nb = in / side;
    return r;
}

struct Plain {};

// ---------------------------------------------------------------- wide

// Warp 0 loads, warp 1 issues MMAs, warps 2-3 prepare scales, warps 4-11 sum
// and store.  Launched with 168 registers a thread (64512 a block); the first
// four warps give some up to the summing ones, which then spill nothing: 128 *
// 152 + 256 * 176 = 64512.
constexpr int kWideThreads = 384;
constexpr int kWideEpi = 8;
constexpr int kChunk = 8;           // K blocks whose scales are prepared at once (32 bytes of a row's)
constexpr int kChunks = 2;

struct Wide {
    static constexpr int N = 256;                           // columns of one tile's sums: two halves of 128
    static constexpr int kTileA = BM * BK;
    static constexpr int kTileB = N / 2 * BK;
    static constexpr int kStageBytes = kTileA + kTileB;
    // (a fifth stage measured level)
    static constexpr int kStages = 4;
    static constexpr int kCols = N;                         // one of two buffers of tensor memory
    static constexpr int kStageY = kWideEpi * 2 * kBox * 64;
    static constexpr int kBars = 2 * kStages + 2 + 2 * kChunks + 1 + 4;
    static constexpr int kScales = kChunks * kChunk * 2 * BM * 4;   // [chunk][K block][half][row]
    static constexpr int kMax = 2 * 2 * BM * 4;             // row maxima of two column halves, two tiles
    static constexpr int kPrefix = (kMaxGroups + 4) * 4;
    static constexpr int kSmemBytes =
        1024 + kStages * kStageBytes + kStageY + kScales + kMax + kBars * 8 + 16 + kPrefix;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory per block");
};

// A tile is 256 rows (128 per block of the pair) and two halves of 128 columns:
// two neighbouring blocks of b's columns (Act = Plain; T is y's 16-bit type), or
// a gate and an up block (y is quantised, T is unused).
// Warps 2-3 fetch the row scales eight K blocks at a time (32 bytes of a row),
// multiply them by the two weight scales and leave the products in shared
// memory, two chunks ahead: loaded by the summing threads one K block ahead,
// their latency was the bound (0.70 PFLOP/s at 4096 x 4096 x 2 x 14336).
template <class Act, class T>
__global__ void __launch_bounds__(kWideThreads, 1)
    gemm_q_wide_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w0,
                       const __grid_constant__ CUtensorMap tm_w1, const __grid_constant__ CUtensorMap tm_y,
                       const Params p)
{
    using S = Wide;
    constexpr int ST = S::kStages;
    constexpr bool kPlain = std::is_same<Act, Plain>::value;
    constexpr int kOutCols = kPlain ? 256 : 128;    // output columns of a tile
    constexpr uint32_t kIdesc = idesc_e4m3(2 * BM, S::kCols);

    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = saddr(smem_raw);
    unsigned char *smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    unsigned char *ystage = smem + ST * S::kStageBytes;
    float *scales = reinterpret_cast<float *>(ystage + S::kStageY);
    float *rowmax = scales + S::kScales / 4;
    uint64_t *full = reinterpret_cast<uint64_t *>(rowmax + S::kMax / 4);
    uint64_t *used = full + ST;             // [ST]: the MMAs of a stage done: it is free and its sums are there
    uint64_t *acc_empty = used + ST;        // [2]: both blocks' epilogues have read a buffer of sums
    uint64_t *sc_full = acc_empty + 2;      // [kChunks]: a chunk of scales is in shared memory
    uint64_t *sc_empty = sc_full + kChunks;
    uint64_t *done = sc_empty + kChunks;    // every MMA of the pair done
    uint64_t *maxbar = done + 1;            // [4]: both column halves of 32 rows have their maxima
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(maxbar + 4);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(maxbar + 4) + 1;
    int *prefix = reinterpret_cast<int *>(maxbar + 6);

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int cluster = blockIdx.x / 2, n_clusters = gridDim.x / 2;

    auto raise_abort = [&]() {
        atomicAdd(&g_q_timeouts, 1u);
        *abort_flag = 1;
        const uint32_t other = mapa(saddr(const_cast<int *>(abort_flag)), rank ^ 1u);
        asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(other), "r"(1) : "memory");
    };

    if (threadIdx.x == 0) {
        const auto init = [](uint64_t *b, uint32_t n) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(n) : "memory");
        };
        for (int s = 0; s < ST; ++s) {
            init(&full[s], 1);
            init(&used[s], 1);
        }
        for (int b = 0; b < 2; ++b) init(&acc_empty[b], kWideEpi * 2);
        for (int b = 0; b < 4; ++b) init(&maxbar[b], 2);
        for (int c = 0; c < kChunks; ++c) {
            init(&sc_full[c], 2);
            init(&sc_empty[c], kWideEpi);
        }
        init(done, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<2>(saddr(const_cast<uint32_t *>(tmem_slot)), 2 * S::kCols);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    count_tiles(p, 2 * BM, prefix);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = *tmem_slot;
    const int n_tiles = prefix[p.n_groups] * p.n_blocks;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 152;");
        if (warp == 0 && lane == 0) {
            uint32_t it = 0;
            for (int t = cluster; t < n_tiles && !*abort_flag; t += n_clusters) {
                const Tile tl = tile_at(p, prefix, t, 2 * BM);
                const int m0 = tl.row + int(rank) * BM;
                // this block's half of the weight rows: 128 columns of y, or gate or up
                const CUtensorMap *tw = rank == 0 ? &tm_w0 : &tm_w1;
                const int w0 = tl.nb * kOutCols + (kPlain ? int(rank) * 128 : 0);
                for (int kt = 0; kt < p.k_tiles; ++kt, ++it) {
                    const uint32_t s = it % ST, use = it / ST;
                    if (*abort_flag) break;
                    if (use > 0 && !wait_parity(saddr(&used[s]), (use - 1) & 1)) {
                        raise_abort();
                        break;
                    }
                    const uint32_t st = saddr(smem + s * S::kStageBytes);
                    // both blocks' copies count on block 0's barrier, which
                    // alone arrives, expecting the bytes of the pair
                    uint32_t bar = saddr(&full[s]);
                    if (rank == 0)
                        arrive_expect_tx_local(bar, uint32_t(2 * S::kStageBytes));
                    else
                        bar = mapa(bar, 0);
                    tma_load<2>(st, &tm_a, kt * BK, m0, bar);
                    tma_load3<2>(st + S::kTileA, tw, kt * BK, w0, tl.e, bar);
                }
            }
            if (rank == 0) {    // the last copies have landed before the block may exit
                const uint32_t first = it > uint32_t(ST) ? it - ST : 0;
                for (uint32_t j = first; j < it; ++j)
                    if (!wait_parity(saddr(&full[j % ST]), (j / ST) & 1)) {
                        atomicAdd(&g_q_timeouts, 1u);
                        break;
                    }
            }
        } else if (warp == 1) {
            // The issuing loop is a bound of its own (it took 860 cycles a K
            // block with one commit for the stage, another for the sums and the
            // abort flag read every time): one barrier tells both the loader
            // and the epilogues that the MMAs of a stage are done.
            if (rank == 0) {
                uint32_t st = 0, phase = 0, ab = 0, acc_phase = 1;     // the first waits on acc_empty pass
                bool ok = true;
                const uint32_t ring = saddr(smem);
                for (int t = cluster; t < n_tiles && ok; t += n_clusters) {
                    for (int kt = 0; kt < p.k_tiles; ++kt) {
                        const uint32_t a0 = ring + st * S::kStageBytes;
                        const uint64_t da = desc_sw128(a0), db = desc_sw128(a0 + S::kTileA);
                        ok = wait_quick(saddr(&full[st]), phase) && wait_quick(saddr(&acc_empty[ab]), acc_phase);
                        ok = __all_sync(0xFFFFFFFFu, ok);
                        if (!ok) {
                            if (lane == 0) raise_abort();
                            break;
                        }
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < BK / 32; ++kk) {
                                const uint64_t step = uint64_t(kk * 32 >> 4);   // 32 bytes inside the swizzle row
                                mma_f8<2>(tmem + ab * S::kCols, da + step, db + step, kIdesc, kk != 0);
                            }
                            mma_commit<2>(saddr(&used[st]));
                        }
                        __syncwarp();
                        if (++st == ST) {
                            st = 0;
                            phase ^= 1;
                        }
                        ab ^= 1;
                        if (ab == 0) acc_phase ^= 1;
                    }
                }
                if (elect_one()) mma_commit<2>(saddr(done));
                __syncwarp();
                // (in block 1 a scale warp waits for this, below: a wait from
                // here would span the whole grid's work, longer than a wait may
                // last, and in the summing warps it would cost them registers)
                if (!wait_parity(saddr(done), 0) && lane == 0) atomicAdd(&g_q_timeouts, 1u);
            }
        } else if (warp >= 2) {
            // scales: this thread prepares two of the block's 128 rows
            const int id = (warp - 2) * 32 + lane;
            uint32_t cc = 0;
            bool ok = true;
            const int wlast = (p.N - 1) / quant::kBlock;
            for (int t = cluster; t < n_tiles && ok; t += n_clusters) {
                const Tile tl = tile_at(p, prefix, t, 2 * BM);
                const int m0 = tl.row + int(rank) * BM + id;
                const float *sa0 = p.sa + int64_t(m0 < tl.end ? m0 : 0) * p.sa_stride;
                const float *sa1 = p.sa + int64_t(m0 + 64 < tl.end ? m0 + 64 : 0) * p.sa_stride;
                const int b0 = kPlain ? tl.nb * 2 : tl.nb, b1 = kPlain ? min(b0 + 1, wlast) : b0;
                const float *sw0 = p.sw0 + int64_t(tl.e) * p.sw_group + int64_t(b0) * p.sw_stride;
                const float *sw1 = p.sw1 + int64_t(tl.e) * p.sw_group + int64_t(b1) * p.sw_stride;
                for (int kb = 0; kb < p.k_tiles; kb += kChunk, ++cc) {
                    float r0[kChunk], r1[kChunk], v0[kChunk], v1[kChunk];
#pragma unroll
                    for (int k = 0; k < kChunk; ++k) {
                        const bool in = kb + k < p.k_tiles;
                        r0[k] = in && m0 < tl.end ? sa0[kb + k] : 0.0f;
                        r1[k] = in && m0 + 64 < tl.end ? sa1[kb + k] : 0.0f;
                        v0[k] = in ? sw0[kb + k] : 0.0f;
                        v1[k] = in ? sw1[kb + k] : 0.0f;
                    }
                    const uint32_t slot = cc % kChunks, use = cc / kChunks;
                    ok = __all_sync(0xFFFFFFFFu,
                                    *abort_flag == 0 &&
                                        (use == 0 || wait_parity(saddr(&sc_empty[slot]), (use - 1) & 1)));
                    if (!ok) {
                        if (lane == 0) raise_abort();
                        break;
                    }
                    float *o = scales + slot * (kChunk * 2 * BM) + id;
#pragma unroll
                    for (int k = 0; k < kChunk; ++k) {
                        o[(2 * k) * BM] = r0[k] * v0[k];
                        o[(2 * k) * BM + 64] = r1[k] * v0[k];
                        o[(2 * k + 1) * BM] = r0[k] * v1[k];
                        o[(2 * k + 1) * BM + 64] = r1[k] * v1[k];
                    }
                    __syncwarp();
                    if (lane == 0) arrive_local(saddr(&sc_full[slot]));
                }
            }
            // two chunks of K blocks are left at most
            if (rank == 1 && warp == 2 && !wait_parity(saddr(done), 0) && lane == 0) atomicAdd(&g_q_timeouts, 1u);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        // warp w reads lanes 32 (w % 4) .. +31, one row per thread; warps 4-7
        // take the first 64 columns of either half, warps 8-11 the others
        const int q = warp & 3, part = (warp - 4) >> 2;
        const uint32_t lane_base = uint32_t(q * 32) << 16;
        const uint32_t empty0 = mapa(saddr(&acc_empty[0]), 0);
        const uint32_t sc0 = saddr(scales) + uint32_t(q * 32 + lane) * 4;
        uint32_t it = 0, cc = 0, n_boxes = 0;
        int lt = 0;
        bool ok = true;
        for (int t = cluster; t < n_tiles && ok; t += n_clusters, ++lt) {
            // The K loop needs no more than the sums, two times 16 columns on
            // their way and a few counters (with 32 at a time registers were
            // spilled, whose loads were a third of the stalls: 213 us instead of
            // 192 at 4096 x 14336 x 4096); which rows and columns these are is
            // asked behind it.
            f2 acc[2][32];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 32; ++j) acc[h][j] = make_float2(0.0f, 0.0f);
            for (int kt = 0; kt < p.k_tiles; ++kt, ++it) {
                if (kt % kChunk == 0) ok = wait_quick(saddr(&sc_full[cc % kChunks]), (cc / kChunks) & 1);
                const uint32_t sc = sc0 + ((cc % kChunks) * kChunk + uint32_t(kt % kChunk)) * (2 * BM * 4);
                const float f0 = ld_shared(sc), f1 = ld_shared(sc + BM * 4);
                if (kt % kChunk == kChunk - 1 || kt + 1 == p.k_tiles) {     // this chunk read
                    __syncwarp();
                    if (lane == 0) arrive_local(saddr(&sc_empty[cc % kChunks]));
                    ++cc;
                }
                ok = __all_sync(0xFFFFFFFFu, ok && wait_quick(saddr(&used[it % ST]), (it / ST) & 1));
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                if (!ok) {
                    if (lane == 0) raise_abort();
                    break;
                }
                // 16 columns are multiplied while the next 16 are on their way
                const uint32_t a0 = tmem + lane_base + (it & 1) * S::kCols + uint32_t(part * 64);
                uint32_t r[2][16];
                const auto add = [](f2 (&a)[32], int at, const uint32_t (&r)[16], float f) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) a[at + j] = fma2(pair(r[2 * j], r[2 * j + 1]), splat(f), a[at + j]);
                };
                tmem_ld16(a0, r[0]);
#pragma unroll
                for (int c = 0; c < 7; ++c) {
                    tmem_wait(r[c & 1]);
                    tmem_ld16(a0 + uint32_t((c + 1) / 4 * 128 + (c + 1) % 4 * 16), r[(c + 1) & 1]);
                    add(acc[c / 4], c % 4 * 8, r[c & 1], c < 4 ? f0 : f1);
                }
                tmem_wait(r[1]);
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                if (elect_one()) arrive_pair(empty0 + 8 * (it & 1));
                add(acc[1], 24, r[1], f1);
            }
            if (!ok || __any_sync(0xFFFFFFFFu, *abort_flag != 0)) break;
            const Tile tl = tile_at(p, prefix, t, 2 * BM);
            const int base = tl.row + int(rank) * BM + q * 32;
            const int m = base + lane;
            const bool on = m < tl.end;

            // Each warp's 32 rows of 64 bytes go through shared memory.  They may
            // leave through the copy engine if all of them are this expert's,
            // or the matrix ends where they end (the engine clips); else the
            // warp writes them row by row, a row's elements side by side.
            const bool box = p.tma_store && (base + kBox <= tl.end || tl.end == p.M);
            const auto store_box = [&](const uint32_t (&w)[16], int n) {
                if (n >= p.N || base >= tl.end) return;
                unsigned char *buf = ystage + ((warp - 4) * 2 + (n_boxes & 1)) * (kBox * 64);
                if (lane == 0 && n_boxes >= 2)      // the box stored from this buffer has been read
                    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                __syncwarp();
                const uint32_t row = saddr(buf) + uint32_t(lane) * 64u, sw = (uint32_t(lane) >> 1) & 3u;
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c)
                    st_shared16(row + ((c ^ sw) << 4), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                if (box) {
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) tma_store(&tm_y, saddr(buf), n, base);
                    ++n_boxes;
                    return;
                }
                __syncwarp();
                const int rows = min(kBox, tl.end - base);
                const uint32_t at = uint32_t(lane) * 2, cols = uint32_t(p.N - n) * (kPlain ? 2 : 1);
                for (int r = 0; r < rows; ++r) {
                    const uint32_t chunk = (at >> 4) ^ ((uint32_t(r) >> 1) & 3u);
                    const uint16_t v = *reinterpret_cast<const uint16_t *>(buf + r * 64 + chunk * 16 + (at & 15));
                    char *dst = p.y + int64_t(base + r) * p.y_stride + int64_t(n) * (kPlain ? 2 : 1) + at;
                    if constexpr (kPlain) {
                        if (at < cols) *reinterpret_cast<uint16_t *>(dst) = v;
                    } else {
                        if (at < cols) dst[0] = char(v & 0xFFu);
                        if (at + 1 < cols) dst[1] = char(v >> 8);
                    }
                }
                __syncwarp();
            };
            if constexpr (kPlain) {
                using Cd = Codec<T>;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int n = tl.nb * kOutCols + (c / 2) * 128 + part * 64 + (c % 2) * 32;
                    uint32_t w[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const f2 v = acc[c / 2][(c % 2) * 16 + j];
                        const float f[2] = {v.x, v.y};
                        w[j] = Cd::put(f);
                    }
                    store_box(w, n);
                }
            } else {
                // y = act(gate) * up over this thread's 64 columns, and the row's maximum over both parts
                float top = 0.0f;
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    gated4<Act>(acc[0][j], acc[1][j], acc[0][j + 1], acc[1][j + 1]);
                    top = fmaxf(fmaxf(top, fmaxf(fabsf(acc[0][j].x), fabsf(acc[0][j].y))),
                                fmaxf(fabsf(acc[0][j + 1].x), fabsf(acc[0][j + 1].y)));
                }
                float *mx = rowmax + (lt & 1) * 2 * BM + q * 32 + lane;
                mx[part * BM] = top;
                __syncwarp();
                if (lane == 0) arrive_local(saddr(&maxbar[q]));
                ok = __all_sync(0xFFFFFFFFu, wait_parity(saddr(&maxbar[q]), lt & 1));
                if (!ok) {
                    if (lane == 0) raise_abort();
                    break;
                }
                top = fmaxf(top, mx[(part ^ 1) * BM]);
                const quant::Divider d(top);
                const f2 inv = splat(d.factor());
                uint32_t w[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const f2 a = mul2(acc[0][2 * j], inv), b = mul2(acc[0][2 * j + 1], inv);
                    w[j] = quant::pack4(a.x, a.y, b.x, b.y);
                }
                if (on && part == 0) p.ys[int64_t(m) * p.ys_stride + tl.nb] = d.scale();
                store_box(w, tl.nb * kOutCols + part * 64);
            }
        }
        if (lane == 0 && n_boxes > 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }

    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    cluster_sync();         // neither block leaves while the other may still signal its barriers
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc<2>(tmem, 2 * S::kCols);
    }
}

// ---------------------------------------------------------------- narrow

constexpr int kNarrowThreads = 192;     // warp 0 loads, warp 1 issues MMAs, warps 2-5 sum and store
constexpr int kAhead = 4;               // K blocks whose row scales are loaded ahead
constexpr int kMaxSplit = 8;            // blocks of a cluster that share a tile's K blocks

constexpr int pow2_at_least(int v) { return v <= 32 ? 32 : v <= 64 ? 64 : v <= 128 ? 128 : v <= 256 ? 256 : 512; }

template <int NT, int MATS>
struct Narrow {
    static constexpr int kTileW = BM * BK;
    static constexpr int kTileA = NT * BK;
    static constexpr int kStageBytes = MATS * kTileW + kTileA;
    static constexpr int kStages = 104 * 1024 / kStageBytes;        // two blocks per SM
    static_assert(kStages >= 3, "stages in flight");
    static constexpr int kCols = MATS * NT;
    static constexpr int kTmemCols = pow2_at_least(2 * kCols);
    static constexpr int kRing = kStages * kStageBytes;
    static constexpr int kParts = MATS * NT * BM * 4;       // one block's sums, for the cluster (over the ring)
    static constexpr int kScl = 4 * 2 * NT * 4;             // row scales, per warp, two K blocks
    static constexpr int kMax = 2 * 4 * NT * 4;             // column maxima of the four warps, two tiles
    static constexpr int kBars = 2 * kStages + 4 + 1 + 1;
    static constexpr int kPrefix = (kMaxGroups + 4) * 4;
    static constexpr int kSmemBytes = 1024 + kRing + kScl + kMax + kBars * 8 + 16 + kPrefix;
    static_assert(kParts <= kRing, "the parts fit the ring");
    static_assert(kTileA % 1024 == 0, "swizzle atoms stay 1024-byte aligned");
    static_assert(kSmemBytes <= 227 * 1024, "shared memory per block");
};

template <class Act, class T, int NT>
__global__ void __launch_bounds__(kNarrowThreads)
    gemm_q_narrow_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w0,
                         const __grid_constant__ CUtensorMap tm_w1, const Params p, const int split)
{
    constexpr bool kPlain = std::is_same<Act, Plain>::value;
    constexpr int MATS = kPlain ? 1 : 2;
    using S = Narrow<NT, MATS>;
    constexpr int ST = S::kStages;
    constexpr uint32_t kIdesc = idesc_e4m3(BM, NT);

    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = saddr(smem_raw);
    unsigned char *smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    float *scl = reinterpret_cast<float *>(smem + S::kRing);            // [4 warps][2][NT]
    float *colmax = scl + 4 * 2 * NT;                                   // [2 tiles][4 warps][NT]
    uint64_t *full = reinterpret_cast<uint64_t *>(colmax + 2 * 4 * NT);
    uint64_t *empty = full + ST;
    uint64_t *acc_full = empty + ST;
    uint64_t *acc_empty = acc_full + 2;
    uint64_t *done = acc_empty + 2;
    uint64_t *maxbar = done + 1;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(maxbar + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(maxbar + 1) + 1;
    int *prefix = reinterpret_cast<int *>(maxbar + 3);
    float *parts = reinterpret_cast<float *>(smem);                     // [MATS * NT][BM], after the last MMA

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = split > 1 ? cluster_rank() : 0u;
    const int cluster = int(blockIdx.x) / split, n_clusters = int(gridDim.x) / split;

    auto raise_abort = [&]() {
        atomicAdd(&g_q_timeouts, 1u);
        *abort_flag = 1;
    };

    if (threadIdx.x == 0) {
        const auto init = [](uint64_t *b, uint32_t n) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(n) : "memory");
        };
        for (int s = 0; s < ST; ++s) {
            init(&full[s], 1);
            init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            init(&acc_full[b], 1);
            init(&acc_empty[b], 4);
        }
        init(done, 1);
        init(maxbar, 4);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<1>(saddr(const_cast<uint32_t *>(tmem_slot)), S::kTmemCols);
    // without experts the block's first weights are known: L2 is asked for a
    // ring of them while the previous kernel ends (L2 is the point of
    // coherence: what that kernel still writes there is read after the wait)
    if (!p.offsets && warp == 2 && lane < ST) {
        const int nb = cluster / p.m_tiles, kt = int(int64_t(p.k_tiles) * rank / split) + lane;
        if (nb < p.n_blocks && kt < p.k_tiles) {
            prefetch3(&tm_w0, kt * BK, nb * BM);
            if constexpr (!kPlain) prefetch3(&tm_w1, kt * BK, nb * BM);
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    count_tiles(p, NT, prefix);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = *tmem_slot;
    const int n_tiles = prefix[p.n_groups] * p.n_blocks;
    // this block's K blocks; with split > 1 a cluster has one tile
    const int k0 = int(int64_t(p.k_tiles) * rank / split), k1 = int(int64_t(p.k_tiles) * (rank + 1) / split);
    const int t_end = split > 1 ? min(n_tiles, cluster + 1) : n_tiles;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            for (int t = cluster; t < t_end && !*abort_flag; t += n_clusters) {
                const Tile tl = tile_at(p, prefix, t, NT);
                for (int kt = k0; kt < k1; ++kt, ++it) {
                    const uint32_t s = it % ST, use = it / ST;
                    if (*abort_flag) break;
                    if (use > 0 && !wait_parity(saddr(&empty[s]), (use - 1) & 1)) {
                        raise_abort();
                        break;
                    }
                    const uint32_t st = saddr(smem + s * S::kStageBytes), bar = saddr(&full[s]);
                    arrive_expect_tx_local(bar, uint32_t(S::kStageBytes));
                    tma_load3<1>(st, &tm_w0, kt * BK, tl.nb * BM, tl.e, bar);
                    if constexpr (!kPlain) tma_load3<1>(st + S::kTileW, &tm_w1, kt * BK, tl.nb * BM, tl.e, bar);
                    tma_load<1>(st + MATS * S::kTileW, &tm_a, kt * BK, tl.row, bar);
                }
            }
            const uint32_t first = it > uint32_t(ST) ? it - ST : 0;
            for (uint32_t j = first; j < it; ++j)
                if (!wait_parity(saddr(&full[j % ST]), (j / ST) & 1)) {
                    atomicAdd(&g_q_timeouts, 1u);
                    break;
                }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = cluster; t < t_end && ok; t += n_clusters) {
                for (int kt = k0; kt < k1; ++kt, ++it) {
                    const uint32_t s = it % ST, use = it / ST;
                    const uint32_t ab = it & 1, use_acc = it >> 1;
                    if (*abort_flag || (use_acc > 0 && !wait_parity(saddr(&acc_empty[ab]), (use_acc - 1) & 1)) ||
                        !wait_parity(saddr(&full[s]), use & 1)) {
                        raise_abort();
                        ok = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t w0 = saddr(smem + s * S::kStageBytes);
                    const uint64_t db = desc_sw128(w0 + MATS * S::kTileW);
#pragma unroll
                    for (int mat = 0; mat < MATS; ++mat) {
                        const uint64_t da = desc_sw128(w0 + mat * S::kTileW);
#pragma unroll
                        for (int kk = 0; kk < BK / 32; ++kk) {
                            const uint64_t step = uint64_t(kk * 32 >> 4);
                            mma_f8<1>(tmem + ab * S::kCols + mat * NT, da + step, db + step, kIdesc, kk != 0);
                        }
                    }
                    mma_commit<1>(saddr(&empty[s]));
                    mma_commit<1>(saddr(&acc_full[ab]));
                }
            }
            mma_commit<1>(saddr(done));
            if (!wait_parity(saddr(done), 0)) atomicAdd(&g_q_timeouts, 1u);
        }
    }

    // ---- sums: one weight row (output column) per thread, NT rows of a
    const int q = warp & 3;
    const bool epi = warp >= 2;
    float acc[MATS][NT];
    // stores rows j0 .. j0 + n - 1 of the tile from sum(mat, j); called by the
    // four epilogue warps
    const auto finish = [&](const Tile &tl, int j0, int n, int lt, auto sum) -> bool {
        const int c = tl.nb * BM + q * 32 + lane;
        if constexpr (kPlain) {
            using Cd = Codec<T>;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (j >= n) break;
                const int m = tl.row + j0 + j;
                if (m < tl.end && c < p.N)
                    Cd::store1(p.y + int64_t(m) * p.y_stride + int64_t(c) * 2, sum(0, j));
            }
            return true;
        } else {
            float y[NT];
            float *mx = colmax + (lt & 1) * 4 * NT;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (j >= n) break;
                y[j] = gated<Act>(splat(sum(0, j)), splat(sum(1, j))).x;
                // magnitudes order like their bits; NaN (above every number) is left out
                const uint32_t b = __float_as_uint(fabsf(y[j]));
                const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, b > 0x7F800000u ? 0u : b);
                if (lane == 0) mx[q * NT + j] = __uint_as_float(top);
            }
            __syncwarp();
            if (lane == 0) arrive_local(saddr(maxbar));
            if (!__all_sync(0xFFFFFFFFu, wait_parity(saddr(maxbar), lt & 1))) {
                if (lane == 0) raise_abort();
                return false;
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (j >= n) break;
                const int m = tl.row + j0 + j;
                if (m >= tl.end) break;
                const quant::Divider d(fmaxf(fmaxf(mx[j], mx[NT + j]), fmaxf(mx[2 * NT + j], mx[3 * NT + j])));
                const float v = y[j] * d.factor();
                if (c < p.N) p.y[int64_t(m) * p.y_stride + c] = char(quant::pack4(v, 0.0f, 0.0f, 0.0f) & 0xFFu);
                if (q == 0 && lane == 0) p.ys[int64_t(m) * p.ys_stride + tl.nb] = d.scale();
            }
            return true;
        }
    };
    bool ok = true;
    if (epi) {
        constexpr int NL = NT > 32 ? NT / 32 : 1;       // row scales per lane
        const uint32_t lane_base = uint32_t(q * 32) << 16;
        float *mine = scl + q * 2 * NT;
        uint32_t it = 0;
        int lt = 0;
        for (int t = cluster; t < t_end && ok; t += n_clusters, ++lt) {
            const Tile tl = tile_at(p, prefix, t, NT);
            const float *s0 = p.sw0 + int64_t(tl.e) * p.sw_group + int64_t(tl.nb) * p.sw_stride;
            const float *s1 = p.sw1 + int64_t(tl.e) * p.sw_group + int64_t(tl.nb) * p.sw_stride;
            const float *sa[NL];
            bool on[NL];
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int j = lane + 32 * i, m = tl.row + j;
                on[i] = j < NT && m < tl.end;
                sa[i] = p.sa + int64_t(on[i] ? m : 0) * p.sa_stride;
            }
#pragma unroll
            for (int mat = 0; mat < MATS; ++mat)
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[mat][j] = 0.0f;
            float na[kAhead][NL], n0[kAhead], n1[kAhead];
            const auto fetch = [&](int slot, int kt) {
                const bool in = kt < k1;
#pragma unroll
                for (int i = 0; i < NL; ++i) na[slot][i] = in && on[i] ? sa[i][kt] : 0.0f;
                n0[slot] = in ? s0[kt] : 0.0f;
                n1[slot] = in && !kPlain ? s1[kt] : 0.0f;
            };
#pragma unroll
            for (int u = 0; u < kAhead; ++u) fetch(u, k0 + u);
            for (int kb = k0; kb < k1 && ok; kb += kAhead) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    if (kb + u >= k1) break;
                    float *sc = mine + (it & 1) * NT;
#pragma unroll
                    for (int i = 0; i < NL; ++i)
                        if (lane + 32 * i < NT) sc[lane + 32 * i] = na[u][i];
                    const float f0 = n0[u], f1 = n1[u];
                    fetch(u, kb + u + kAhead);
                    __syncwarp();
                    const uint32_t ab = it & 1, use_acc = it >> 1;
                    ok = __all_sync(0xFFFFFFFFu, wait_parity(saddr(&acc_full[ab]), use_acc & 1));
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    if (!ok) {
                        if (lane == 0) raise_abort();
                        break;
                    }
                    const uint32_t a0 = tmem + lane_base + ab * S::kCols;
#pragma unroll
                    for (int c = 0; c < NT; c += 16) {
                        uint32_t r0[16], r1[16];
                        tmem_ld16(a0 + uint32_t(c), r0);
                        if constexpr (!kPlain) {
                            tmem_ld16(a0 + uint32_t(NT + c), r1);
                            tmem_wait(r1);
                        }
                        tmem_wait(r0);
                        if (c + 16 == NT) {
                            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                            __syncwarp();
                            if (lane == 0) arrive_local(saddr(&acc_empty[ab]));
                        }
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 s4 = *reinterpret_cast<const float4 *>(sc + c + j);
                            const float sv[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                acc[0][c + j + i] = fmaf(__uint_as_float(r0[j + i]), sv[i] * f0, acc[0][c + j + i]);
                                if constexpr (!kPlain)
                                    acc[MATS - 1][c + j + i] =
                                        fmaf(__uint_as_float(r1[j + i]), sv[i] * f1, acc[MATS - 1][c + j + i]);
                            }
                        }
                    }
                    ++it;
                }
            }
            if (!ok || split > 1) break;
            if (__any_sync(0xFFFFFFFFu, *abort_flag != 0)) break;
            ok = finish(tl, 0, NT, lt, [&](int mat, int j) { return acc[mat][j]; });
        }
    }

    if (split > 1) {
        // the parts of the blocks of the cluster, added in the order of their
        // ranks; block r finishes rows NT / split * r .. of the tile
        const bool has = cluster < n_tiles;
        if (epi && has) {
            const int row = q * 32 + lane;
#pragma unroll
            for (int mat = 0; mat < MATS; ++mat)
#pragma unroll
                for (int j = 0; j < NT; ++j) parts[(mat * NT + j) * BM + row] = acc[mat][j];
        }
        cluster_sync();
        if (epi && has) {
            bool all = true;
            for (int r = 0; r < split; ++r) {
                const uint32_t flag = mapa(saddr(const_cast<int *>(abort_flag)), uint32_t(r));
                all = all && __float_as_int(ld_cluster(flag)) == 0;
            }
            if (__all_sync(0xFFFFFFFFu, all)) {
                const Tile tl = tile_at(p, prefix, cluster, NT);
                const int n = NT / split, j0 = int(rank) * n;
                finish(tl, j0, n, 0, [&](int mat, int j) {
                    // (all loads before the first sum: each is a trip to another SM)
                    const uint32_t at = saddr(parts + (mat * NT + j0 + j) * BM + q * 32 + lane);
                    float v[kMaxSplit], sum = 0.0f;
#pragma unroll
                    for (int r = 0; r < kMaxSplit; ++r) v[r] = r < split ? ld_cluster(mapa(at, uint32_t(r))) : 0.0f;
#pragma unroll
                    for (int r = 0; r < kMaxSplit; ++r) sum += v[r];
                    return sum;
                });
            }
        }
        cluster_sync();     // no block leaves while another may still read its parts
    }

    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc<1>(tmem, S::kTmemCols);
    }
}

// K == 0: empty sums, so zeros (and the scale of a block of zeros) in every row
// of every expert.
__global__ void gemm_q_zero_kernel(const Params p, int out_bytes)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int lo = 0, hi = p.M;
    if (p.offsets) {
        lo = min(max(p.offsets[0], 0), p.M);
        hi = min(max(p.offsets[p.n_groups], lo), p.M);
    }
    const int64_t width = int64_t(p.N) * out_bytes;
    for (int64_t m = lo + int64_t(blockIdx.x); m < hi; m += gridDim.x) {
        for (int64_t c = threadIdx.x; c < width; c += blockDim.x) p.y[m * p.y_stride + c] = 0;
        if (p.ys)
            for (int c = threadIdx.x; c <= (p.N - 1) / quant::kBlock; c += blockDim.x)
                p.ys[m * p.ys_stride + c] = quant::kAmaxFloor / quant::kFp8Max;
    }
}

cudaError_t timeouts(unsigned int *count, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(count, g_q_timeouts, sizeof(unsigned int));
    if (e == cudaSuccess && reset) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_q_timeouts, &zero, sizeof(unsigned int));
    }
    return e;
}

// ---------------------------------------------------------------- host side

namespace {

// A row-major byte (or 16-bit, for y) matrix, or a stack of them, as a tensor
// map; loads read zeros outside it and stores drop what falls outside.
bool make_map(CUtensorMap *m, CUtensorMapDataType type, const void *base, int64_t cols, int64_t rows,
              int64_t stride_bytes, int64_t depth, int64_t depth_bytes, int box_cols, int box_rows,
              CUtensorMapSwizzle swizzle)
{
    EncodeFn fn = encode_fn();
    if (!fn) return false;
    const int rank = depth > 0 ? 3 : 2;
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(depth)};
    const cuuint64_t strides[2] = {cuuint64_t(stride_bytes), cuuint64_t(depth_bytes)};
    const cuuint32_t box[3] = {cuuint32_t(box_cols), cuuint32_t(box_rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, type, cuuint32_t(rank), const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Output of a call: 0-3 the gated activations (8-bit y), 4 f16, 5 bf16.
constexpr int kOutF16 = 4, kOutBF16 = 5;

using WideFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, Params);
using NarrowFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, Params, int);

WideFn wide_kernel(int out)
{
    using B = __nv_bfloat16;
    switch (out) {
    case 0: return gemm_q_wide_kernel<Silu, B>;
    case 1: return gemm_q_wide_kernel<GeluErf, B>;
    case 2: return gemm_q_wide_kernel<GeluTanh, B>;
    case 3: return gemm_q_wide_kernel<Relu, B>;
    case 4: return gemm_q_wide_kernel<Plain, __half>;
    default: return gemm_q_wide_kernel<Plain, B>;
    }
}

NarrowFn narrow_kernel(int out, int nt, int *smem)
{
    using B = __nv_bfloat16;
    using H = __half;
    *smem = out < kOutF16 ? Narrow<16, 2>::kSmemBytes
            : nt == 16    ? Narrow<16, 1>::kSmemBytes
            : nt == 32    ? Narrow<32, 1>::kSmemBytes
                          : Narrow<64, 1>::kSmemBytes;
    switch (out) {
    case 0: return gemm_q_narrow_kernel<Silu, B, 16>;
    case 1: return gemm_q_narrow_kernel<GeluErf, B, 16>;
    case 2: return gemm_q_narrow_kernel<GeluTanh, B, 16>;
    case 3: return gemm_q_narrow_kernel<Relu, B, 16>;
    case kOutF16:
        return nt == 16   ? gemm_q_narrow_kernel<Plain, H, 16>
               : nt == 32 ? gemm_q_narrow_kernel<Plain, H, 32>
                          : gemm_q_narrow_kernel<Plain, H, 64>;
    default:
        return nt == 16   ? gemm_q_narrow_kernel<Plain, B, 16>
               : nt == 32 ? gemm_q_narrow_kernel<Plain, B, 32>
                          : gemm_q_narrow_kernel<Plain, B, 64>;
    }
}

// The shared-memory opt-in of each kernel, once per device.
constexpr int kMaxDevices = 64;
std::atomic<int> g_opted[kMaxDevices][6][4];    // [device][output][wide, 16, 32, 64]

int opt_in(const void *fn, int smem, int dev, int out, int shape)
{
    std::atomic<int> &f = g_opted[dev % kMaxDevices][out][shape];
    if (dev < kMaxDevices && f.load(std::memory_order_acquire)) return GLU_OK;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return glu::cuda_fail(e);
    }
    f.store(1, std::memory_order_release);
    return GLU_OK;
}

int launch(const void *fn, unsigned grid, unsigned threads, int smem, unsigned cluster, void **args,
           cudaStream_t stream)
{
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
    if (e != cudaSuccess) {     // retry without the dependent-launch attribute
        (void)cudaGetLastError();
        cfg.attrs = &attr[1];
        cfg.numAttrs = cluster > 1 ? 1 : 0;
        e = cudaLaunchKernelExC(&cfg, fn, args);
    }
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return glu::cuda_fail(e);
    }
    return GLU_OK;
}

struct Args {
    const void *a;
    int64_t a_stride;
    const float *sa;
    int64_t sa_stride;
    const void *w0, *w1;
    int64_t w_stride, w_group;
    const float *sw0, *sw1;
    int64_t sw_stride, sw_group;
    void *y;
    int64_t y_stride;
    float *ys;
    int64_t ys_stride;
    int64_t M, K, N;
    const int32_t *offsets;
    int64_t groups;             // 0: dense
    int out;
};

// The bytes of a stack of `depth` matrices, `group` elements apart; none for empty matrices.
bool stack_span(const void *q, int64_t rows, int64_t stride, int64_t cols, int64_t group, int64_t depth, int e, Span *o)
{
    if (!span(q, rows, stride, cols, e, o)) return false;
    int64_t more = 0;
    return depth <= 1 || o->lo == o->hi ||
           (!__builtin_mul_overflow(group, int64_t(e), &more) && !__builtin_mul_overflow(more, depth - 1, &more) &&
            !__builtin_add_overflow(o->hi, uint64_t(more), &o->hi));
}

// Argument rules shared by the four entry points; no CUDA call.
int validate(Args &x, bool *empty)
{
    *empty = false;
    const bool plain = x.out >= kOutF16;
    if (x.M < 0 || x.K < 0 || x.N < 0 || x.groups < 0 || x.M > INT32_MAX - 65536 || x.K > INT32_MAX - 65536 ||
        x.N > INT32_MAX - 65536 || x.groups > kMaxGroups)
        return GLU_ERR_SHAPE;
    if (x.M == 0 || x.N == 0 || (x.offsets == nullptr && x.groups > 0 && x.M == 0)) {
        *empty = true;
        return GLU_OK;
    }
    const bool grouped = x.groups > 0;
    if (!x.y || (!plain && !x.ys) || (grouped && !x.offsets)) return GLU_ERR_NULL;
    if (x.K > 0 && (!x.a || !x.sa || !x.w0 || !x.w1 || !x.sw0 || !x.sw1)) return GLU_ERR_NULL;
    const int64_t kb = (x.K + quant::kBlock - 1) / quant::kBlock, nb = (x.N + quant::kBlock - 1) / quant::kBlock;
    const int64_t depth = grouped ? x.groups : 1;
    const int E = plain ? 2 : 1;
    if (x.M == 1) {
        x.sa_stride = kb;
        x.y_stride = x.y_stride < x.N ? x.N : x.y_stride;
        x.ys_stride = nb;
    }
    // strides that separate nothing
    if (nb == 1) x.sw_stride = kb;
    if (x.N == 1) x.w_stride = (x.K + 15) / 16 * 16;
    if (depth == 1) x.w_group = x.sw_group = 0;
    if (x.y_stride < x.N || (!plain && x.ys_stride < nb)) return GLU_ERR_STRIDE;
    if (x.K > 0) {
        if (x.M == 1) x.a_stride = (x.K + 15) / 16 * 16;
        if (x.a_stride < x.K || x.w_stride < x.K || x.sa_stride < kb || x.sw_stride < kb) return GLU_ERR_STRIDE;
        // the tensor-memory accelerator needs 16-byte aligned bases and strides (below 2^40 bytes)
        if (uintptr_t(x.a) % 16 || uintptr_t(x.w0) % 16 || uintptr_t(x.w1) % 16 || x.a_stride % 16 ||
            x.w_stride % 16 || x.a_stride >= (int64_t(1) << 40) || x.w_stride >= (int64_t(1) << 40))
            return GLU_ERR_STRIDE;
        if (grouped && (x.w_group % 16 || x.w_group >= (int64_t(1) << 40))) return GLU_ERR_STRIDE;
        if (uintptr_t(x.sa) % 4 || uintptr_t(x.sw0) % 4 || uintptr_t(x.sw1) % 4) return GLU_ERR_STRIDE;
    }
    if ((plain && uintptr_t(x.y) % 2) || (!plain && uintptr_t(x.ys) % 4) || uintptr_t(x.offsets) % 4)
        return GLU_ERR_STRIDE;
    Span s[9] = {};
    int64_t wspan = 0, swspan = 0;
    if (grouped && x.K > 0) {
        if (x.w_group < 0 || x.sw_group < 0) return GLU_ERR_STRIDE;
        if (__builtin_mul_overflow(x.N - 1, x.w_stride, &wspan) || __builtin_add_overflow(wspan, x.K, &wspan) ||
            __builtin_mul_overflow(nb - 1, x.sw_stride, &swspan) || __builtin_add_overflow(swspan, kb, &swspan))
            return GLU_ERR_SHAPE;
        if (depth > 1 && (x.w_group < wspan || x.sw_group < swspan)) return GLU_ERR_STRIDE;
    }
    const auto stack = [&](const void *q, int64_t rows, int64_t stride, int64_t cols, int64_t group, int e, Span *o) {
        return stack_span(q, rows, stride, cols, group, depth, e, o);
    };
    bool fits = span(x.y, x.M, x.y_stride, x.N, E, &s[0]) &&
                span(x.ys, plain ? 0 : x.M, x.ys_stride, nb, 4, &s[1]) &&
                span(x.offsets, grouped ? 1 : 0, 1, x.groups + 1, 4, &s[2]);
    if (x.K > 0)
        fits = fits && span(x.a, x.M, x.a_stride, x.K, 1, &s[3]) && span(x.sa, x.M, x.sa_stride, kb, 4, &s[4]) &&
               stack(x.w0, x.N, x.w_stride, x.K, x.w_group, 1, &s[5]) &&
               stack(x.w1, x.N, x.w_stride, x.K, x.w_group, 1, &s[6]) &&
               stack(x.sw0, nb, x.sw_stride, kb, x.sw_group, 4, &s[7]) &&
               stack(x.sw1, nb, x.sw_stride, kb, x.sw_group, 4, &s[8]);
    if (!fits) return GLU_ERR_SHAPE;
    if (overlap(s[0], s[1])) return GLU_ERR_ALIAS;
    for (int o = 0; o < 2; ++o)
        for (int i = 2; i < 9; ++i)
            if (overlap(s[o], s[i])) return GLU_ERR_ALIAS;
    return GLU_OK;
}

// The operands of the tensor-memory accelerator are in the current device's
// memory.
int check_device(const Args &x)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    for (const void *q : {x.a, x.w0, x.w1 == x.w0 ? nullptr : x.w1, static_cast<const void *>(x.y)}) {
        if (!q || (x.K == 0 && q != x.y)) continue;
        cudaPointerAttributes at{};
        if (e == cudaSuccess) e = cudaPointerGetAttributes(&at, q);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return glu::cuda_fail(e);
        }
        if (at.type != cudaMemoryTypeDevice || at.device != dev) return GLU_ERR_VALUE;
    }
    return GLU_OK;
}

int run(Args x, glu_stream_t stream)
{
    bool empty = false;
    if (int st = validate(x, &empty)) return st;
    if (empty) {
        glu::record_launch(glu_launch_info_t{});
        return GLU_OK;
    }
    const bool plain = x.out >= kOutF16, grouped = x.groups > 0;
    const int E = plain ? 2 : 1;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (int st = check_device(x)) return st;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return glu::cuda_fail(e);
    }
    Params p{};
    p.sa = x.sa;
    p.sa_stride = x.sa_stride;
    p.sw0 = x.sw0;
    p.sw1 = x.sw1;
    p.sw_stride = x.sw_stride;
    p.sw_group = x.sw_group;
    p.y = static_cast<char *>(x.y);
    p.y_stride = x.y_stride * E;
    p.ys = x.ys;
    p.ys_stride = x.ys_stride;
    p.offsets = grouped ? x.offsets : nullptr;
    p.n_groups = grouped ? int(x.groups) : 1;
    p.M = int(x.M);
    p.N = int(x.N);
    p.k_tiles = int((x.K + BK - 1) / BK);
    glu_launch_info_t info{};
    info.launched = 1;
    info.path = plain ? 12 : 11;
    if (x.K == 0) {
        int out_bytes = E;
        void *args[] = {&p, &out_bytes};
        const unsigned grid = unsigned(x.M < 8 * sms ? x.M : 8 * sms);
        if (int st = launch(reinterpret_cast<const void *>(&gemm_q_zero_kernel), grid, 256, 0, 1, args, s)) return st;
        info.threads = 256;
        info.grid = int32_t(grid);
        glu::record_launch(info);
        return GLU_OK;
    }

    const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const int64_t depth = grouped ? x.groups : 1;
    const int64_t w_group = grouped && depth > 1 ? x.w_group : (x.N * x.w_stride + 15) / 16 * 16;
    // rows per expert, as far as the host knows
    const int64_t rows = grouped ? (x.M + x.groups - 1) / x.groups : x.M;
    CUtensorMap ta, t0, t1, ty;
    // rows a narrow tile takes: 16, 32 or 64 for the plain product; always 16 for
    // the gated one, whose tiles of 32 leave room for one block per SM only (200
    // rows, 8 experts of 4096 x 14336: 186 us with tiles of 16, 226 with 32; one
    // MLP and 32 rows: 28.4, 30.5)
    const int nt = rows <= 16 || !plain ? 16 : rows <= 32 ? 32 : 64;
    const int64_t n_blocks = (x.N + BM - 1) / BM;
    // row tiles; with experts at most: each may end in a part of a tile
    const auto row_tiles = [&](int64_t r) {
        return grouped ? x.M / r + (x.groups < x.M ? x.groups : x.M) : (x.M + r - 1) / r;
    };
    const int64_t tiles_n = row_tiles(nt) * n_blocks;
    const int64_t slots_n = int64_t(sms) * 2;
    // Narrow: blocks per tile, the split of K whose rounds of tiles take the
    // least time: in K blocks, a round costs about ten more for its start and
    // its end, and adding the parts half a one each.  (By expert only where the
    // most tiles there can be have their parts on the GPU at once: a split grid
    // holds a cluster for each of them, with a tile or not.)
    int split = 1;
    int64_t best = -1;
    for (int sp = 1; sp <= kMaxSplit && (sp == 1 || sp * 2 <= p.k_tiles); sp *= 2) {
        if (sp > 1 && grouped && tiles_n * sp > slots_n) break;
        const int64_t cost = (tiles_n * sp + slots_n - 1) / slots_n * ((p.k_tiles + sp - 1) / sp + 10) + sp / 2;
        if (best < 0 || cost < best) {
            best = cost;
            split = sp;
        }
    }
    // Which kernel.  Up to 32 rows the narrow one wins throughout (16 rows at
    // 4096 x 4096: 7.2 us against 19).  Beyond, the gated product is wide (64
    // rows at 4096 x 14336: 36 us against 54 in narrow tiles of 16); the plain
    // one is narrow by expert up to 96 rows each (64 experts of 2048 x 2048: 73
    // us against 87 at 64 rows, 108 against 96 at 128), else where its rounds, of
    // K blocks that take 4/3 the wide kernel's time, end sooner (14336 x 4096:
    // 24 us against 56 at 128 rows, 41 against 57 at 256, 69 against 58 at 384).
    const int64_t tiles_w = row_tiles(2 * BM) * ((x.N + (plain ? 255 : 127)) / (plain ? 256 : 128));
    const int64_t cost_w = (tiles_w + sms / 2 - 1) / (sms / 2) * (p.k_tiles + 9);
    const bool narrow = rows <= 32 || (plain && (grouped ? rows <= 96 : 4 * best / 3 < cost_w));
    if (narrow) {
        const int64_t m_tiles = row_tiles(nt);
        if (tiles_n > INT32_MAX / 16) return GLU_ERR_SHAPE;
        p.n_blocks = int(n_blocks);
        p.m_tiles = p.group_m = int(m_tiles);
        if (!make_map(&ta, u8, x.a, x.K, x.M, x.a_stride, 0, 0, BK, nt, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !make_map(&t0, u8, x.w0, x.K, x.N, x.w_stride, depth, w_group, BK, BM, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !make_map(&t1, u8, x.w1, x.K, x.N, x.w_stride, depth, w_group, BK, BM, CU_TENSOR_MAP_SWIZZLE_128B))
            return glu::cuda_fail(cudaErrorInvalidValue);
        int smem = 0;
        const void *f = reinterpret_cast<const void *>(narrow_kernel(x.out, nt, &smem));
        if (int st = opt_in(f, smem, dev, x.out, nt == 16 ? 1 : nt == 32 ? 2 : 3)) return st;
        const int64_t grid = split > 1 ? tiles_n * split : (tiles_n < slots_n ? tiles_n : slots_n);
        void *args[] = {&ta, &t0, &t1, &p, &split};
        if (int st = launch(f, unsigned(grid), kNarrowThreads, smem, unsigned(split), args, s)) return st;
        info.threads = kNarrowThreads;
        info.grid = int32_t(grid);
        info.unroll = split;
        info.vec_bytes = E;
        info.vector_units = grouped ? 0 : tiles_n;
        glu::record_launch(info);
        return GLU_OK;
    }

    const int out_cols = plain ? 256 : 128;
    p.n_blocks = int((x.N + out_cols - 1) / out_cols);
    const int64_t block_bytes = int64_t(2 * BM) * x.K;
    int64_t group = (int64_t(48) << 20) / block_bytes;
    group = group < 1 ? 1 : group;
    const int64_t m_tiles = row_tiles(2 * BM);
    if (group > m_tiles) group = m_tiles;
    const int64_t tiles = tiles_w;
    if (tiles > INT32_MAX / 16) return GLU_ERR_SHAPE;
    p.m_tiles = int(m_tiles);
    p.group_m = int(group);
    if (!make_map(&ta, u8, x.a, x.K, x.M, x.a_stride, 0, 0, BK, BM, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&t0, u8, x.w0, x.K, x.N, x.w_stride, depth, w_group, BK, BM, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map(&t1, u8, x.w1, x.K, x.N, x.w_stride, depth, w_group, BK, BM, CU_TENSOR_MAP_SWIZZLE_128B))
        return glu::cuda_fail(cudaErrorInvalidValue);
    const auto yt = x.out == kOutF16    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                    : x.out == kOutBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                        : u8;
    // the copy engine clips a box at y's last column in 16-byte units
    p.tma_store = uintptr_t(x.y) % 16 == 0 && p.y_stride % 16 == 0 && (x.N * E) % 16 == 0 && p.y_stride < (int64_t(1) << 40) &&
                  make_map(&ty, yt, x.y, x.N, x.M, p.y_stride, 0, 0, 64 / E, kBox, CU_TENSOR_MAP_SWIZZLE_64B);
    if (!p.tma_store) ty = ta;
    const int smem = Wide::kSmemBytes;
    const void *f = reinterpret_cast<const void *>(wide_kernel(x.out));
    if (int st = opt_in(f, smem, dev, x.out, 0)) return st;
    const int64_t slots = sms / 2;
    const int64_t clusters = tiles < slots ? tiles : slots;
    void *args[] = {&ta, &t0, &t1, &ty, &p};
    if (int st = launch(f, unsigned(2 * clusters), kWideThreads, smem, 2, args, s)) return st;
    info.threads = kWideThreads;
    info.grid = int32_t(2 * clusters);
    info.unroll = 2;
    info.vec_bytes = p.tma_store ? 64 : E;
    info.vector_units = grouped ? 0 : tiles;
    glu::record_launch(info);
    return GLU_OK;
}

}  // namespace
}  // namespace gemmq
}  // namespace glu

extern "C" int glu_gemm_q_nt(const void *a, int64_t a_stride, const float *a_scale, int64_t a_scale_stride,
                             const void *b, int64_t b_stride, const float *b_scale, int64_t b_scale_stride, void *d,
                             int64_t d_stride, int64_t M, int64_t K, int64_t N, glu_dtype_t dtype, glu_stream_t stream)
{
    using namespace glu::gemmq;
    if (dtype != GLU_F16 && dtype != GLU_BF16) return GLU_ERR_ENUM;
    return run({a, a_stride, a_scale, a_scale_stride, b, b, b_stride, 0, b_scale, b_scale, b_scale_stride, 0, d,
                d_stride, nullptr, 0, M, K, N, nullptr, 0, dtype == GLU_F16 ? kOutF16 : kOutBF16},
               stream);
}

extern "C" int glu_gemm_q_fwd(const void *x, int64_t x_stride, const float *x_scale, int64_t x_scale_stride,
                              const void *w_gate, const void *w_up, int64_t w_stride, const float *gate_scale,
                              const float *up_scale, int64_t w_scale_stride, void *y, int64_t y_stride,
                              float *y_scale, int64_t y_scale_stride, int64_t M, int64_t K, int64_t I, glu_act_t act,
                              glu_stream_t stream)
{
    using namespace glu::gemmq;
    if (act < GLU_ACT_SILU || act > GLU_ACT_RELU) return GLU_ERR_ENUM;
    return run({x, x_stride, x_scale, x_scale_stride, w_gate, w_up, w_stride, 0, gate_scale, up_scale, w_scale_stride,
                0, y, y_stride, y_scale, y_scale_stride, M, K, I, nullptr, 0, int(act)},
               stream);
}

extern "C" int glu_gemm_q_grouped_nt(const void *a, int64_t a_stride, const float *a_scale, int64_t a_scale_stride,
                                     const void *b, int64_t b_stride, int64_t b_group, const float *b_scale,
                                     int64_t b_scale_stride, int64_t b_scale_group, void *d, int64_t d_stride,
                                     int64_t M, int64_t K, int64_t N, const int32_t *offsets, int64_t n_groups,
                                     glu_dtype_t dtype, glu_stream_t stream)
{
    using namespace glu::gemmq;
    if (dtype != GLU_F16 && dtype != GLU_BF16) return GLU_ERR_ENUM;
    if (n_groups == 0) M = 0;           // no expert, so no row
    return run({a, a_stride, a_scale, a_scale_stride, b, b, b_stride, b_group, b_scale, b_scale, b_scale_stride,
                b_scale_group, d, d_stride, nullptr, 0, M, K, N, offsets, n_groups,
                dtype == GLU_F16 ? kOutF16 : kOutBF16},
               stream);
}

extern "C" int glu_gemm_q_grouped_fwd(const void *x, int64_t x_stride, const float *x_scale, int64_t x_scale_stride,
                                      const void *w_gate, const void *w_up, int64_t w_stride, int64_t w_group,
                                      const float *gate_scale, const float *up_scale, int64_t w_scale_stride,
                                      int64_t w_scale_group, void *y, int64_t y_stride, float *y_scale,
                                      int64_t y_scale_stride, int64_t M, int64_t K, int64_t I, const int32_t *offsets,
                                      int64_t n_groups, glu_act_t act, glu_stream_t stream)
{
    using namespace glu::gemmq;
    if (act < GLU_ACT_SILU || act > GLU_ACT_RELU) return GLU_ERR_ENUM;
    if (n_groups == 0) M = 0;
    return run({x, x_stride, x_scale, x_scale_stride, w_gate, w_up, w_stride, w_group, gate_scale, up_scale,
                w_scale_stride, w_scale_group, y, y_stride, y_scale, y_scale_stride, M, K, I, offsets, n_groups,
                int(act)},
               stream);
}

// ---------------------------------------------------------------- the gated MLP

namespace glu {
namespace gemmq {
namespace {

int64_t round_up16(int64_t v) { return (v + 15) / 16 * 16; }

}  // namespace
}  // namespace gemmq
}  // namespace glu

extern "C" size_t glu_mlp_q_workspace_bytes(int64_t M, int64_t I)
{
    using namespace glu::gemmq;
    if (M <= 0 || I <= 0 || M > INT32_MAX || I > INT32_MAX) return 0;
    return size_t(M) * size_t(round_up16(I) + (I + glu::quant::kBlock - 1) / glu::quant::kBlock * 4);
}

extern "C" int glu_mlp_q_fwd(const void *x, int64_t x_stride, const float *x_scale, int64_t x_scale_stride,
                             const void *w_gate, const void *w_up, int64_t w_stride, int64_t w_group,
                             const float *gate_scale, const float *up_scale, int64_t w_scale_stride,
                             int64_t w_scale_group, const void *w_down, int64_t w_down_stride, int64_t w_down_group,
                             const float *down_scale, int64_t down_scale_stride, int64_t down_scale_group, void *out,
                             int64_t out_stride, int64_t M, int64_t H, int64_t I, const int32_t *offsets,
                             int64_t n_groups, glu_act_t act, glu_dtype_t dtype, void *workspace,
                             size_t workspace_bytes, glu_stream_t stream)
{
    using namespace glu::gemmq;
    if (act < GLU_ACT_SILU || act > GLU_ACT_RELU || (dtype != GLU_F16 && dtype != GLU_BF16)) return GLU_ERR_ENUM;
    if (!offsets)
        n_groups = 0;
    else if (n_groups == 0 && M > 0)    // no expert, so no row
        M = 0;
    if (M < 0 || H < 0 || I < 0 || M > INT32_MAX || I > INT32_MAX) return GLU_ERR_SHAPE;
    if (M > 0 && H > 0 && I > 0) {
        if (!workspace || workspace_bytes < glu_mlp_q_workspace_bytes(M, I)) return GLU_ERR_WORKSPACE;
        if (uintptr_t(workspace) % 16) return GLU_ERR_STRIDE;
    }
    // the workspace: y's rows of round_up(I, 16) bytes, then its scales
    const int64_t ys = round_up16(I), groups = (I + glu::quant::kBlock - 1) / glu::quant::kBlock;
    float *y_scale = I > 0 && workspace ? reinterpret_cast<float *>(static_cast<char *>(workspace) + M * ys) : nullptr;
    Args up{x, x_stride, x_scale, x_scale_stride, w_gate, w_up, w_stride, w_group, gate_scale, up_scale,
            w_scale_stride, w_scale_group, workspace, ys, y_scale, groups, M, H, I, offsets, n_groups, int(act)};
    Args down{workspace, ys, y_scale, groups, w_down, w_down, w_down_stride, w_down_group, down_scale, down_scale,
              down_scale_stride, down_scale_group, out, out_stride, nullptr, 0, M, I, H, offsets, n_groups,
              dtype == GLU_F16 ? kOutF16 : kOutBF16};
    if (H == 0) up.M = down.M = 0;
    // both calls are checked before the first launch
    Args cu = up, cd = down;
    bool empty = false;
    if (I > 0)
        if (int st = validate(cu, &empty)) return st;
    if (int st = validate(cd, &empty)) return st;
    if (!empty) {
        // out and the whole workspace against every operand of either product
        const int64_t hb = (H + glu::quant::kBlock - 1) / glu::quant::kBlock, depth = n_groups > 1 ? n_groups : 1;
        const int64_t used = I > 0 ? 1 : 0;         // I == 0 reads and writes none of them
        glu::Span outs[2] = {}, in[9] = {};
        const bool fits =
            glu::span(out, M, cd.y_stride, H, 2, &outs[0]) &&
            glu::span(workspace, used, 1, M * (ys + 4 * groups), 1, &outs[1]) &&
            glu::span(x, used * M, cu.a_stride, H, 1, &in[0]) &&
            glu::span(x_scale, used * M, cu.sa_stride, hb, 4, &in[1]) &&
            stack_span(w_gate, used * I, cu.w_stride, H, cu.w_group, depth, 1, &in[2]) &&
            stack_span(w_up, used * I, cu.w_stride, H, cu.w_group, depth, 1, &in[3]) &&
            stack_span(gate_scale, used * groups, cu.sw_stride, hb, cu.sw_group, depth, 4, &in[4]) &&
            stack_span(up_scale, used * groups, cu.sw_stride, hb, cu.sw_group, depth, 4, &in[5]) &&
            stack_span(w_down, used * H, cd.w_stride, I, cd.w_group, depth, 1, &in[6]) &&
            stack_span(down_scale, used * hb, cd.sw_stride, groups, cd.sw_group, depth, 4, &in[7]) &&
            glu::span(offsets, n_groups > 0 ? 1 : 0, 1, n_groups + 1, 4, &in[8]);
        if (!fits) return GLU_ERR_SHAPE;
        if (glu::overlap(outs[0], outs[1])) return GLU_ERR_ALIAS;
        for (const glu::Span &o : outs)
            for (const glu::Span &i : in)
                if (glu::overlap(o, i)) return GLU_ERR_ALIAS;
        if (I > 0)
            if (int st = check_device(cu)) return st;
        if (int st = check_device(cd)) return st;
        if (I > 0)
            if (int st = run(up, stream)) return st;
    }
    return run(down, stream);
}
