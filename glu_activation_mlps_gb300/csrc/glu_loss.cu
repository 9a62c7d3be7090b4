// Losses over a vocabulary straight from the hidden rows x (N x H) and the output
// projection w (V x H), on the fifth-generation tensor cores of sm_103a.  With
// z = x w^T, s = z / T (T = 1 for the cross entropy), lse = log sum_v exp s_v:
//
//     cross entropy   loss = lse - z_target
//     distillation    loss = sum_k p_k (log p_k - s_{index k} + lse),  p = softmax over k of t_k / T
//     gradient        g_v  = dloss / T (exp(s_v - lse) - [target share of v])
//                     dx   = g w,   dw = g^T x
//
// The logits are not kept between the passes.  The forward product's epilogue
// reduces each tile of them to a maximum and a sum per row and picks the few logits
// the loss names; the backward pass forms them again, a piece of the vocabulary at a
// time, and its epilogue turns them into g in 16 bits, which the two gradient
// products read.  Sums are fp32 throughout.
//
// g rounds to the inputs' type because one tensor-core product takes one type: half
// a step, relative 2^-8 or 2^-11 an entry; up to 64 rows in two parts (g_parts, which
// has the price of a second part and what one costs).  It is formed with the largest
// |dloss| / T at a power of two, put back in fp32: the share at a target is then within
// p of -1 of it for p below half a step, whatever number of rows a mean divides by (8192 rows of
// which 3277 have a target, against 64 bits in the 2-norm: dx and dw off by 2.2e-3 ->
// 1.85e-3, 1.7e-3 of it their own rounding), and shares of 1 / V are normal f16 numbers.
//
// One kernel template runs the four products (stats, grad, data, weight) on the
// structure of glu_gemm.cu: a persistent grid; warp 0 fills a ring of 64-deep K
// slices with the tensor-memory accelerator (128-byte swizzle), one thread of
// warp 1 issues tcgen05.mma into one of two accumulators, and two warpgroups add
// the other one, a segment of K, to the sums in their registers.  The operands lie
// as the user has them: g w wants w's vocabulary as its K, g^T x wants rows as K,
// so those come as MN-major tiles (64 columns x 64 K to a swizzled box), which the
// MMA reads directly.  Only x is transposed in memory, where dw is large.
//
// Bound: the tensor cores (large calls run at the power limit, 1.6 - 1.75 PFLOP/s,
// where the library's plain bf16 product settles at 1.7), w's bytes (few rows, 5.3
// - 5.8 TB/s) or launches (a small forward call is two of 5 us).
//
// Rows without a target take no part in any product: a first kernel lists the
// rows that have one and, only where some have none, copies them side by side.
// The count stays on the device; the grids are sized for all rows and their
// tiles counted in the kernel.
//
// Waits are bounded as in glu_gemm.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "glu.h"
#include "glu_kernels.cuh"
#include "glu_internal.h"
#include "glu_tensor.cuh"

namespace glu {
namespace loss {

using namespace glu::gemm;

constexpr int BM = 128;                 // rows of a tile per block (tensor-memory lanes)
constexpr int BK = 64;                  // K per stage: 64 x 2 bytes = one 128-byte swizzle row
constexpr int kThreads = 384;           // warp 0 loads, warp 1 issues MMAs, warps 4-11 take the sums
constexpr int kEpiWarps = 8;            // 32 rows each, in two halves of the columns
// Registers of a thread: launched with 168 (65536 over 384 threads); warps 0-3
// give theirs up to 72, the others take 216 for a row's 128 sums and what forms
// the results: 128 x 72 + 256 x 216 = 384 x 168.  Tiles of 256 columns spill all the
// same (44 - 136 bytes stored and 120 - 228 loaded a thread), narrower ones 16 bytes or
// nothing.
constexpr int kRegsLaunch = 168, kRegsFew = 72, kRegsMany = 216;
static_assert(128 * kRegsFew + 256 * kRegsMany <= kThreads * kRegsLaunch, "the split fits the launch");
constexpr int kRingBytes = 192 * 1024;
constexpr int kBoxBytes = 4096;         // results leave through boxes of 32 rows x 128 bytes, one a warp
constexpr int kChunkBytes = 64 * BK * 2;    // an MN-major box: 64 columns x 64 K
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

enum Mode {
    kStats,     // z = x w^T -> per tile and row: maximum, sum of exponentials, named logits
    kGrad,      // z = x w^T -> g
    kData,      // g w     (K = the piece's vocabulary)
    kWeight,    // g^T x   (K = rows)
    kWeightT    // the same with x transposed before (K-major)
};
__host__ __device__ constexpr bool is_weight(int mode) { return mode == kWeight || mode == kWeightT; }
__host__ __device__ constexpr bool is_gradient(int mode) { return mode == kData || is_weight(mode); }

template <int MODE, int BN, int CTAS>
struct Shape {
    static constexpr bool kTransA = is_weight(MODE);
    static constexpr bool kTransB = MODE == kData || MODE == kWeight;
    static constexpr int kTileN = 2 * BN;                               // columns of a tile
    static constexpr int kBRows = CTAS == 1 ? 2 * BN : BN;              // of them, loaded by one block
    static constexpr int kTileA = BM * BK * 2;
    // dx of up to 64 rows: a stage holds both parts of g for one slice of w, the second in
    // the tile's upper half.  One MMA reads the tile from its start, a second from the middle
    // on; what that makes of the accumulator's upper 64 rows is no row of dx.
    static constexpr int kAParts = MODE == kData && CTAS == 1 ? 2 : 1;
    static constexpr int kSecondA = kTileA / 2;
    static constexpr int kTileB = kBRows * BK * 2;
    static constexpr int kStageBytes = kTileA + kTileB;
    static constexpr int kStages = kRingBytes / kStageBytes > 8 ? 8 : kRingBytes / kStageBytes;
    static constexpr int kTileM = BM * CTAS;
    static constexpr int kTmemCols = 2 * kTileN <= 256 ? 256 : 512;     // two accumulators, a power of two
    static constexpr int kBars = 2 * kStages + 2 + 2 + 1;               // full, empty, acc_full, acc_empty, done
    static constexpr int kStageOut = is_gradient(MODE) ? kEpiWarps * kBoxBytes : 0;
    static constexpr int kCols = kTileN / 2;                            // columns of one epilogue thread
    // K slices summed in tensor memory before their sum goes to registers.  The forward pass:
    // 768 products, where the logits are off as much as fp32 products on the ordinary cores
    // (1024 x 4096, 32768 tokens, 2-norm against 64 bits: segments of 1024 9.9e-7 in 161 us, of
    // 768 7.0e-7 in 163, of 512 4.7e-7 in 165, fp32 6.1e-7; 4096 x 4096, 131072: 2268, 2302, 2336
    // us).  For few rows, whose time is w's bytes, 128 (loss of one row, 1024 x 8192, median of 40:
    // of 256 1.6e-7 in 10.0 us, of 128 1.0e-7 in 10.6, fp32 1.0e-7; 64 rows, 4096 x 32768: 48.7 and
    // 48.8 us).  What is rounded to 16 bits takes longer ones.
    static constexpr int kSegment = is_gradient(MODE) ? 64 / kAParts
                                    : MODE == kStats  ? (CTAS == 2 ? 12 : 2)
                                                      : (CTAS == 2 ? 16 : 4);
    static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kStageOut + kBars * 8 + 16;
    static_assert(BN % 32 == 0 && BN >= 32 && kTileN <= 256, "one MMA covers the tile's columns");
    static_assert(!kTransB || kBRows % 64 == 0, "MN-major operands come in chunks of 64 columns");
    static_assert(kTileA % 1024 == 0 && kTileB % 1024 == 0, "swizzle atoms stay 1024-byte aligned");
    static_assert(kSmemBytes <= 227 * 1024, "shared memory per block");
};

// The last tiles of a gradient's product, which would leave most of the GPU idle
// for a round, are cut along K: tiles from `whole` on into `parts` parts each,
// whose fp32 sums are kept apart (part q of tile whole + i is number q * tail +
// i) and added in their order by sum_kernel.
struct Cut {
    int whole, parts;
};

struct Params {
    const int *count;           // rows that take part; rows[] lists them
    const int *rows;
    int N;                      // rows of x
    int copied;                 // the listed rows are copied even if they are all
    int cols;                   // columns of the output: the piece's vocabulary (stats, grad), H (data, weight)
    int depth;                  // K: H (stats, grad), the piece's vocabulary (data); weight: the count
    int m_rows;                 // rows of the output for weight: the piece's vocabulary
    int n_blocks;
    const Cut *cut;             // data, weight
    int group_m;                // row blocks per group of the tile order
    uint32_t a_bytes;           // bytes of A in a stage (stats, grad, data: rows that exist, up to 128)
    // stats
    float2 *part;               // [2 n_blocks][N]: maximum (in log2 units) and sum of half a tile's columns
    float *named;               // cross entropy: the target's logit by listed row; distillation: [N][top] by row
    const int64_t *target;      // cross entropy
    const int *index;           // distillation: [N][top], sorted, INT_MAX where there is none
    int top;
    int64_t first;              // first token of the piece
    float c1;                   // log2(e) / T
    // grad
    const float *lse, *loss, *dloss;
    float inv_t;
    const float *scale;         // [0] what g is scaled by, [1] its inverse
    // grad, data, weight
    int parts;                  // 16-bit parts of g
    int part_cols;              // columns of g from the first to the second
    // data, weight
    char *out;
    int64_t out_stride;         // bytes
    int vec_store;              // rows are 32- or 16-byte aligned; 0: at any place
    int tma_store;              // results may leave through boxes
    int sums;                   // fp32 sums of this piece instead of results: 1 stored, 2 added to the last piece's
};

static __device__ unsigned int g_loss_timeouts;

// Shared-memory matrix descriptor of an MN-major tile, 128-byte swizzle: atoms
// of 64 columns x 8 K (1024 bytes); the stride byte offset is the step of 8 K,
// the leading byte offset the step of 64 columns.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t addr)
{
    uint64_t d = 0;
    d |= uint64_t((addr & 0x3FFFF) >> 4);
    d |= uint64_t(kChunkBytes >> 4) << 16;
    d |= uint64_t(1024 >> 4) << 32;
    d |= uint64_t(1) << 46;
    d |= uint64_t(2) << 61;
    return d;
}

__device__ __forceinline__ void tma_add(const CUtensorMap *map, uint32_t src, int x, int y)
{
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

__device__ __forceinline__ void tma_prefetch(const CUtensorMap *map, int x, int y)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y)
                 : "memory");
}

// An arrival on the other block's barrier that hands back tensor memory.  What it
// orders, the tensor-memory reads, is complete (wait::ld); a release to the cluster
// would wait for this thread's global stores of the tile before as well.
__device__ __forceinline__ void arrive_remote(uint32_t bar_cluster)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

__device__ __forceinline__ float exp2_fast(float v)
{
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// 32 values of 16 bits to 64 bytes of a row, 32-byte aligned.
__device__ __forceinline__ void store_row(char *dst, const uint32_t (&w)[16])
{
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const uint32_t w8[8] = {w[8 * v],     w[8 * v + 1], w[8 * v + 2], w[8 * v + 3],
                                w[8 * v + 4], w[8 * v + 5], w[8 * v + 6], w[8 * v + 7]};
        Access<32>::store(dst + 32 * v, w8);
    }
}

__device__ __forceinline__ f2 pair(const uint32_t (&g)[32], int j)
{
    return make_float2(__uint_as_float(g[j]), __uint_as_float(g[j + 1]));
}

// Element j of a row's 32 registers, j known at run time only.
__device__ __forceinline__ float pick(const uint32_t (&g)[32], int j)
{
    uint32_t v = g[0];
#pragma unroll
    for (int i = 1; i < 32; ++i) v = j == i ? g[i] : v;
    return __uint_as_float(v);
}

// Tile t: row block and column block.
struct Tile {
    int mb, nb;
};

__device__ __forceinline__ Tile tile_of(int group_m, int n_blocks, int t, int m_blocks)
{
    const int per_group = group_m * n_blocks;
    const int first_m = (t / per_group) * group_m;
    const int gsize = min(m_blocks - first_m, group_m);
    const int r = t % per_group;
    return {first_m + r % gsize, r / gsize};
}

constexpr int kMaxParts = 16;
constexpr int kTailRounds = 4;          // tail parts: at most this many rounds of the GPU

// The cheapest cut, counted in slices of K of a slot, a round costing 8 more to
// start and to store; parts of 4 slices at least.  No cut for less than 4 %.  Lane
// s tries s parts, of the last round's tiles or of the last two rounds'.
__device__ __forceinline__ Cut cut_of(int tiles, int k_tiles, int slots, int lane)
{
    const int rem = tiles % slots;
    const uint32_t none = uint32_t((tiles + slots - 1) / slots) * uint32_t(k_tiles + 8);
    uint32_t cost = UINT32_MAX;
    int whole = tiles;
    // no part without a slice: so many parts that the last would start behind K are left out
    const bool full = lane >= 2 && (lane - 1) * ((k_tiles + lane - 1) / lane) < k_tiles;
    if (rem != 0 && full && lane <= kMaxParts && k_tiles >= 4 * lane && tiles < 26 * slots) {
        for (int tail = rem; tail <= tiles && tail <= rem + slots && tail * lane <= kTailRounds * slots; tail += slots) {
            const uint32_t v = uint32_t((tiles - tail) / slots) * uint32_t(k_tiles + 8) +
                               uint32_t((tail * lane + slots - 1) / slots) * uint32_t((k_tiles + lane - 1) / lane + 8);
            if (v < cost) {
                cost = v;
                whole = tiles - tail;
            }
        }
    }
    const uint32_t best = __reduce_min_sync(0xFFFFFFFFu, cost);
    if (best >= none - none / 25) return {tiles, 1};
    const int from = __ffs(__ballot_sync(0xFFFFFFFFu, cost == best)) - 1;
    return {__shfl_sync(0xFFFFFFFFu, whole, from), from};
}

// A block's work item: its tile, the slices of K, and its number among the parts
// kept apart (-1: none).
struct Item {
    Tile tile;
    int k0, n_k, part;
};

template <int MODE, class T, int BN, int CTAS>
__global__ void __launch_bounds__(kThreads, 1)
    loss_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_listed, const __grid_constant__ CUtensorMap tm_out,
                     const __grid_constant__ CUtensorMap tm_tail, const Params p)
{
    using S = Shape<MODE, BN, CTAS>;
    using Cd = Codec<T>;
    constexpr int ST = S::kStages;
    constexpr uint32_t kIdesc = idesc_f16(std::is_same<T, __nv_bfloat16>::value ? 1 : 0, S::kTileM, S::kTileN) |
                                (S::kTransA ? 1u << 15 : 0u) | (S::kTransB ? 1u << 16 : 0u);

    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = saddr(smem_raw);
    unsigned char *smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    unsigned char *ostage = smem + ST * S::kStageBytes;                 // 1024-byte aligned
    uint64_t *full = reinterpret_cast<uint64_t *>(ostage + S::kStageOut);
    uint64_t *empty = full + ST;
    uint64_t *acc_full = empty + ST;
    uint64_t *acc_empty = acc_full + 2;
    uint64_t *done = acc_empty + 2;
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(done + 1) + 1;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CTAS == 1 ? 0u : cluster_rank();
    const int cluster = blockIdx.x / CTAS, n_clusters = gridDim.x / CTAS;

    auto raise_abort = [&]() {
        atomicAdd(&g_loss_timeouts, 1u);
        *abort_flag = 1;
        if constexpr (CTAS == 2) {
            const uint32_t other = mapa(saddr(const_cast<int *>(abort_flag)), rank ^ 1u);
            asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(other), "r"(1) : "memory");
        }
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(saddr(&full[s])) : "memory");
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(saddr(&empty[s])) : "memory");
        }
        for (int b = 0; b < 2; ++b) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(saddr(&acc_full[b])) : "memory");
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(&acc_empty[b])),
                         "r"(kEpiWarps * CTAS)
                         : "memory");
        }
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(saddr(done)) : "memory");
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<CTAS>(saddr(const_cast<uint32_t *>(tmem_slot)), S::kTmemCols);
    // few rows: the first tile's rows of w are asked of L2 before the wait for the
    // kernel before (which may still write them: L2 then holds what it wrote)
    if constexpr (CTAS == 1 && (MODE == kStats || MODE == kGrad)) {
        if (warp == 0 && lane == 0 && cluster < p.n_blocks)
            for (int kt = 0; kt < min(ST, (p.depth + BK - 1) / BK); ++kt)
                tma_prefetch(&tm_b, kt * BK, (MODE == kGrad ? p.n_blocks - 1 - cluster : cluster) * S::kTileN);
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    if constexpr (CTAS == 2)
        cluster_sync();
    else
        __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = *tmem_slot;
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // What depends on how many rows take part.  With none there is still one
    // block of rows (or one slice of K): it reads zeros and gives zeros.
    const int count = p.count ? *reinterpret_cast<const volatile int *>(p.count) : p.N;
    const bool all = count == p.N, listed = !all || p.copied;
    const int m_rows = is_weight(MODE) ? p.m_rows : count;
    const int m_blocks = max(1, (m_rows + S::kTileM - 1) / S::kTileM);
    const int parts = is_weight(MODE) ? p.parts : 1;        // slices of g with one slice of x, in turn along K
    const int k_tiles = parts * max(1, ((is_weight(MODE) ? count : p.depth) + BK - 1) / BK);
    const int n_tiles = m_blocks * p.n_blocks;
    const Cut cut = is_gradient(MODE) ? *p.cut : Cut{n_tiles, 1};
    const int tail = n_tiles - cut.whole, per_part = (k_tiles + cut.parts - 1) / cut.parts;
    const int n_items = cut.whole + tail * cut.parts;
    const auto item_of = [&](int t) {
        Item o;
        o.part = t < cut.whole ? -1 : t - cut.whole;
        const int q = o.part < 0 ? 0 : o.part / tail;
        o.tile = tile_of(p.group_m, p.n_blocks, t - q * tail, m_blocks);
        // g walks the vocabulary backwards: the forward pass before left its end in L2
        // (with dx before dw, 3 % of a step of 64 x 4096, 32768 tokens)
        if constexpr (MODE == kGrad) o.tile.nb = p.n_blocks - 1 - o.tile.nb;
        o.k0 = q * per_part;
        o.n_k = o.part < 0 ? k_tiles : min(per_part, k_tiles - o.k0);
        return o;
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
        if (warp == 0) {
            if (lane == 0) {
                const CUtensorMap *ma = (MODE == kStats || MODE == kGrad) && listed ? &tm_listed : &tm_a;
                const CUtensorMap *mbp = MODE == kWeight && listed ? &tm_listed : &tm_b;
                const uint32_t bytes = p.a_bytes + uint32_t(S::kTileB);
                uint32_t it = 0;
                for (int t = cluster; t < n_items && !*abort_flag; t += n_clusters) {
                    const Item o = item_of(t);
                    const int m0 = o.tile.mb * S::kTileM + int(rank) * BM;
                    const int n0 = o.tile.nb * S::kTileN + int(rank) * (CTAS == 1 ? 0 : BN);
                    for (int kt = 0; kt < o.n_k; ++kt, ++it) {
                        const uint32_t s = it % ST, use = it / ST;
                        if (*abort_flag) break;
                        if (use > 0 && !wait_parity(saddr(&empty[s]), (use - 1) & 1)) {
                            raise_abort();
                            break;
                        }
                        const uint32_t st = saddr(smem + s * S::kStageBytes);
                        const bool second = parts == 2 && ((o.k0 + kt) & 1);
                        const int k = (parts == 2 ? (o.k0 + kt) >> 1 : o.k0 + kt) * BK;
                        // both blocks' copies count on block 0's barrier
                        uint32_t bar = saddr(&full[s]);
                        if (rank == 0)
                            arrive_expect_tx_local(bar, bytes * CTAS);
                        else
                            bar = mapa(bar, 0);
                        if constexpr (S::kTransA) {
#pragma unroll
                            for (int c = 0; c < BM / 64; ++c)
                                tma_load<CTAS>(st + c * kChunkBytes, ma, m0 + (second ? p.part_cols : 0) + 64 * c, k,
                                               bar);
                        } else {
                            tma_load<CTAS>(st, ma, k, m0, bar);
                            if constexpr (S::kAParts == 2)
                                if (p.parts == 2) tma_load<CTAS>(st + S::kSecondA, &tm_listed, k, m0, bar);
                        }
                        if constexpr (S::kTransB) {
#pragma unroll
                            for (int c = 0; c < S::kBRows / 64; ++c)
                                tma_load<CTAS>(st + S::kTileA + c * kChunkBytes, mbp, n0 + 64 * c, k, bar);
                        } else {
                            tma_load<CTAS>(st + S::kTileA, mbp, k, n0, bar);
                        }
                    }
                }
                // block 0 holds the barriers of every copy of the pair: wait for the
                // last ones to land before the block may exit
                if (rank == 0) {
                    const uint32_t first = it > uint32_t(ST) ? it - ST : 0;
                    for (uint32_t j = first; j < it; ++j)
                        if (!wait_parity(saddr(&full[j % ST]), (j / ST) & 1)) {
                            atomicAdd(&g_loss_timeouts, 1u);
                            break;
                        }
                }
            }
        } else if (warp == 1) {
            if (lane == 0 && rank == 0) {
                uint32_t it = 0;
                int use = 0;                // accumulators filled so far
                for (int t = cluster; t < n_items && !*abort_flag; t += n_clusters) {
                    const int n_k = item_of(t).n_k;
                    bool ok = true;
                    for (int kt = 0; kt < n_k; ++use) {
                        const int ab = use & 1, use_acc = use >> 1, end = min(n_k, kt + S::kSegment);
                        if (*abort_flag) {
                            ok = false;
                            break;
                        }
                        if (use_acc > 0 && !wait_parity(saddr(&acc_empty[ab]), (use_acc - 1) & 1)) {
                            raise_abort();
                            ok = false;
                            break;
                        }
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        const uint32_t d = tmem + uint32_t(ab * S::kTileN);
                        for (bool more = false; kt < end; ++kt, ++it, more = true) {
                            const uint32_t s = it % ST;
                            if (!wait_parity(saddr(&full[s]), (it / ST) & 1)) {
                                raise_abort();
                                ok = false;
                                break;
                            }
                            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                            const uint32_t a0 = saddr(smem + s * S::kStageBytes);
                            const uint64_t da = S::kTransA ? desc_mn_sw128(a0) : desc_sw128(a0);
                            const uint64_t db = S::kTransB ? desc_mn_sw128(a0 + S::kTileA) : desc_sw128(a0 + S::kTileA);
#pragma unroll
                            for (int kk = 0; kk < BK / 16; ++kk) {
                                // 16 K further: 32 bytes inside the swizzle row, or two
                                // 1024-byte atoms of an MN-major tile
                                const uint64_t sa = uint64_t(kk * (S::kTransA ? 2048 : 32) >> 4);
                                const uint64_t sb = uint64_t(kk * (S::kTransB ? 2048 : 32) >> 4);
                                mma<CTAS>(d, da + sa, db + sb, kIdesc, more || kk != 0);
                                if constexpr (S::kAParts == 2)
                                    if (p.parts == 2) mma<CTAS>(d, da + sa + (S::kSecondA >> 4), db + sb, kIdesc, 1);
                            }
                            mma_commit<CTAS>(saddr(&empty[s]));
                        }
                        if (!ok) break;
                        mma_commit<CTAS>(saddr(&acc_full[ab]));
                    }
                    if (!ok) break;
                }
                mma_commit<CTAS>(saddr(done));
                if (!wait_parity(saddr(done), 0)) atomicAdd(&g_loss_timeouts, 1u);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMany));
        // epilogue: warp w reads tensor-memory lanes 32 (w % 4) .. +31, one row per
        // thread, half of the columns.  The sums of each segment of K are added to
        // the thread's registers: the tensor core's own fp32 sums drop bits towards
        // zero at every step, an error that grows with the steps in one accumulator.
        const int q = warp & 3, col0 = ((warp - 4) >> 2) * S::kCols;
        const uint32_t lane_base = uint32_t(q * 32) << 16;
        const uint32_t boxes = saddr(ostage) + uint32_t(warp - 4) * kBoxBytes;
        bool boxed = false;             // a box of this warp is with the copy engine
        float unscale = 1.0f, gscale = 1.0f;
        if constexpr (MODE == kGrad) gscale = p.scale[0];
        if constexpr (is_gradient(MODE)) unscale = p.scale[1];
        int use = 0;
        bool ok = true;
        for (int t = cluster; t < n_items; t += n_clusters) {
            const Item o = item_of(t);
            const int n_seg = (o.n_k + S::kSegment - 1) / S::kSegment;
            const int m = o.tile.mb * S::kTileM + int(rank) * BM + q * 32 + lane;
            const int n0 = o.tile.nb * S::kTileN + col0;    // this thread's first column
            const bool live = m < m_rows;
            // what this row needs, requested before the wait for its sums
            int row = m;
            int64_t tgt = -1;           // its target, from the first column
            float coef = 0.0f, shift = 0.0f, at_target = 0.0f;
            int e = 0, next = INT32_MAX;
            if constexpr (MODE == kStats || MODE == kGrad) {
                if (live) {
                    if (!all) row = p.rows[m];
                    if (p.target) tgt = p.target[row] - p.first - n0;
                }
            }
            if constexpr (MODE == kStats) {
                if (p.index && live) {
                    // the first of the row's sorted tokens that is not before this column
                    const int *list = p.index + int64_t(row) * p.top;
                    int hi = p.top;
                    while (e < hi) {
                        const int mid = (e + hi) >> 1;
                        if (list[mid] < n0)
                            e = mid + 1;
                        else
                            hi = mid;
                    }
                    if (e < p.top) next = list[e];
                }
            }
            if constexpr (MODE == kGrad) {
                if (live) {
                    coef = p.dloss[row] * p.inv_t * gscale;    // in this order: scale / T may overflow
                    shift = -p.lse[row] * kLog2e;
                    // p - 1 at the target, without the cancellation (the loss is good to its own size)
                    if (p.target && coef != 0.0f) at_target = coef * expm1f(-p.loss[row]);
                }
            }
            if constexpr (MODE == kData) {
                if (live && !all) row = p.rows[m];
            }
            __syncwarp();
            constexpr int kChunks = S::kCols / 32;
            uint32_t sums[kChunks][32];
            for (int seg = 0; seg < n_seg; ++seg, ++use) {
                const int ab = use & 1, use_acc = use >> 1;
                // tcgen05.ld is warp-collective: the whole warp takes one decision
                ok = !__any_sync(0xFFFFFFFFu, *abort_flag != 0);
                if (!ok) break;
                ok = __all_sync(0xFFFFFFFFu, wait_parity_sleep(saddr(&acc_full[ab]), use_acc & 1));
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                if (!ok) {
                    if (lane == 0) raise_abort();
                    break;
                }
                const uint32_t acc = tmem + lane_base + uint32_t(ab * S::kTileN + col0);
                if (seg == 0) {
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) tmem_ld32(acc + uint32_t(32 * c), sums[c]);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                } else {
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        uint32_t g[32];
                        tmem_ld32(acc + uint32_t(32 * c), g);
                        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            const f2 v = add2(pair(sums[c], j), pair(g, j));
                            sums[c][j] = __float_as_uint(v.x);
                            sums[c][j + 1] = __float_as_uint(v.y);
                        }
                    }
                }
                // all of it read: hand the accumulator back
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CTAS == 1)
                        arrive_local(saddr(&acc_empty[ab]));
                    else
                        arrive_remote(mapa(saddr(&acc_empty[ab]), 0));
                }
            }
            if (!ok) break;
            if constexpr (MODE == kStats) {
                const int width = p.cols - n0;              // columns that exist
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    uint32_t (&g)[32] = sums[c];
                    // the target's logit counts in the maximum, but its term is left out of the sum:
                    // beside it the other terms of a confident row would lose the bits that are its loss
                    if (tgt >= 32 * c && tgt < 32 * c + 32) {
                        const int at = int(tgt) - 32 * c;
                        const float z = pick(g, at);
                        p.named[m] = z;
                        top = fmaxf(top, z);
#pragma unroll
                        for (int j = 0; j < 32; ++j) g[j] = at == j ? 0xFF800000u : g[j];
                    }
                    while (next < n0 + 32 * c + 32) {
                        p.named[int64_t(row) * p.top + e] = pick(g, next - n0 - 32 * c);
                        ++e;
                        next = e < p.top ? p.index[int64_t(row) * p.top + e] : INT32_MAX;
                    }
                    __syncwarp();
                    if (width < 32 * c + 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) g[j] = 32 * c + j < width ? g[j] : 0xFF800000u;    // -inf
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) top = fmaxf(top, __uint_as_float(g[j]));
                }
                // maximum (the target's logit included) and sum of exponentials, in units of log2
                top *= p.c1;
                const float base = top == -INFINITY ? 0.0f : top;
                const f2 c1 = splat(p.c1), shift2 = splat(-base);
                f2 s[2] = {splat(0.0f), splat(0.0f)};
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const f2 v = fma2(pair(sums[c], j), c1, shift2);
                        s[j / 2 & 1] = add2(s[j / 2 & 1], make_float2(exp2_fast(v.x), exp2_fast(v.y)));
                    }
                s[0] = add2(s[0], s[1]);
                if (live)
                    p.part[int64_t(2 * o.tile.nb + (col0 != 0)) * p.N + m] = make_float2(top, s[0].x + s[0].y);
            } else {
                const int m_box = m - lane;
                const bool floats = is_gradient(MODE) && (o.part >= 0 || p.sums);
                // 32 columns of a row, rounded
                const auto round16 = [&](int c, uint32_t (&packed)[16]) {
                    const uint32_t (&g)[32] = sums[c];
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        float f[2] = {__uint_as_float(g[j]), __uint_as_float(g[j + 1])};
                        if constexpr (is_gradient(MODE)) {
                            const f2 v = mul2(pair(g, j), splat(unscale));
                            f[0] = v.x;
                            f[1] = v.y;
                        }
                        packed[j / 2] = Cd::put(f);
                    }
                };
                // grad: 32 columns of g in place of their logits
                const auto to_g = [&](int c) {
                    uint32_t (&g)[32] = sums[c];
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const f2 v = fma2(pair(g, j), splat(p.c1), splat(shift));
                        const f2 e = mul2(splat(coef), make_float2(exp2_fast(v.x), exp2_fast(v.y)));
                        g[j] = __float_as_uint(e.x);
                        g[j + 1] = __float_as_uint(e.y);
                    }
                    if (tgt >= 32 * c && tgt < 32 * c + 32) {
                        const int at = int(tgt) - 32 * c;
#pragma unroll
                        for (int j = 0; j < 32; ++j) g[j] = at == j ? __float_as_uint(at_target) : g[j];
                    }
                    // 0 past the piece, and in rows without a gradient, whatever their logits are
                    const int exist = coef == 0.0f ? 0 : p.cols - (n0 + 32 * c);
                    if (exist < 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) g[j] = j < exist ? g[j] : 0u;
                    }
                };
                // A box: row `lane` is 128 bytes, its 16-byte chunk v at v ^ (lane % 8).  The
                // copy engine has read what was there before; then it gets this one.
                const auto box_free = [&]() {
                    if (lane == 0 && boxed) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    boxed = true;
                    __syncwarp();
                };
                const auto to_box = [&](uint32_t v, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
                    st_shared16(boxes + uint32_t(lane) * 128u + ((v ^ (uint32_t(lane) & 7u)) << 4), w0, w1, w2, w3);
                };
                const auto box_full = [&]() {
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                };
                if (floats) {               // fp32 sums, 32 columns to a box
                    const CUtensorMap *map = o.part < 0 ? &tm_out : &tm_tail;
                    const int y = o.part < 0 ? m_box : o.part * S::kTileM + (m_box - o.tile.mb * S::kTileM);
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        const uint32_t (&g)[32] = sums[c];
                        if (n0 + 32 * c >= p.cols) continue;
                        box_free();
#pragma unroll
                        for (uint32_t v = 0; v < 8; ++v) to_box(v, g[4 * v], g[4 * v + 1], g[4 * v + 2], g[4 * v + 3]);
                        box_full();
                        if (lane == 0) {
                            const int x = o.part < 0 ? n0 + 32 * c : col0 + 32 * c;
                            if (p.sums == 2)
                                tma_add(map, boxes, x, y);
                            else
                                tma_store(map, boxes, x, y);
                        }
                    }
                    continue;
                }
                // 16 bits, 64 columns to a box: whole lines, and the fence a box costs is cheaper
                // than the lines that a warp's own stores to 32 rows touch (g and dw of 64 rows,
                // 32768 x 4096: 116 -> 111 us; of 100 rows, 50001 x 1000, rows of 2000 bytes: 80 ->
                // 59).  g itself, whose rows start on lines, is 3 % faster without (300 x 1024,
                // 16384 tokens).
                if (is_gradient(MODE) && kChunks % 2 == 0 && p.tma_store && (MODE != kData || all)) {
#pragma unroll
                    for (int c = 0; c + 1 < kChunks; c += 2) {
                        if (n0 + 32 * c >= p.cols) continue;
                        uint32_t lo[16], hi[16];
                        round16(c, lo);
                        round16(c + 1, hi);
                        box_free();
#pragma unroll
                        for (uint32_t v = 0; v < 4; ++v) {
                            to_box(v, lo[4 * v], lo[4 * v + 1], lo[4 * v + 2], lo[4 * v + 3]);
                            to_box(v + 4, hi[4 * v], hi[4 * v + 1], hi[4 * v + 2], hi[4 * v + 3]);
                        }
                        box_full();
                        if (lane == 0) tma_store(&tm_out, boxes, n0 + 32 * c, m_box);
                    }
                    continue;
                }
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const int left = p.cols - (n0 + 32 * c);    // columns that exist
                    if (left <= 0) continue;
                    uint32_t packed[16];
                    if constexpr (MODE == kGrad) to_g(c);
                    round16(c, packed);
                    char *dst = p.out + int64_t(MODE == kGrad ? m : row) * p.out_stride + int64_t(n0 + 32 * c) * 2;
                    if constexpr (MODE == kGrad) {
                        if (m < p.N) store_row(dst, packed);    // whole chunks: a row of g has room for them
                        if constexpr (CTAS == 1) {              // what the rounding leaves, rounded
                            if (p.parts == 2) {
#pragma unroll
                                for (int j = 0; j < 32; j += 2) {
                                    const float f[2] = {__uint_as_float(sums[c][j]) - Cd::get(packed[j / 2], 0),
                                                        __uint_as_float(sums[c][j + 1]) - Cd::get(packed[j / 2], 1)};
                                    packed[j / 2] = Cd::put(f);
                                }
                                if (m < p.N) store_row(dst + int64_t(p.part_cols) * 2, packed);
                            }
                        }
                        continue;
                    }
                    if (p.vec_store) {
                        if (!live) continue;
                        if (left >= 32 && p.vec_store == 32) {
                            store_row(dst, packed);
                            continue;
                        }
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            const uint32_t w4[4] = {packed[4 * v], packed[4 * v + 1], packed[4 * v + 2],
                                                    packed[4 * v + 3]};
                            if (8 * v + 8 <= left) {
                                Access<16>::store(dst + 16 * v, w4);
                            } else {
#pragma unroll
                                for (int j = 8 * v; j < 8 * v + 8; ++j)
                                    if (j < left) Cd::store1(dst + j * 2, Cd::get(packed[j / 2], j % 2));
                            }
                        }
                        continue;
                    }
                    // rows at any place: through shared memory, 32 values of a row to one access
                    // of the warp (tiles that leave through boxes come after these, if at all)
                    const uint32_t at = boxes + uint32_t(lane) * 68u;
                    __syncwarp();
#pragma unroll
                    for (int v = 0; v < 16; ++v)
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 4u * v), "r"(packed[v]) : "memory");
                    __syncwarp();
                    const int rows_here = min(32, m_rows - m_box);
                    for (int r = 0; r < rows_here; ++r) {
                        const uint64_t to = __shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(dst), r);
                        unsigned short v;
                        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(boxes + uint32_t(r) * 68u + 2u * lane));
                        if (lane < left) asm volatile("st.global.b16 [%0], %1;" ::"l"(to + 2 * lane), "h"(v) : "memory");
                    }
                }
            }
        }
        // every box this warp stored has left shared memory and reached global memory
        if (lane == 0 && boxed) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        if (rank == 1 && warp == 4 && !wait_parity(saddr(done), 0) && lane == 0) atomicAdd(&g_loss_timeouts, 1u);
        __syncwarp();
    }

    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    if constexpr (CTAS == 2)
        cluster_sync();
    else
        __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc<CTAS>(tmem, S::kTmemCols);
    }
}

// ---------------------------------------------------------------- the small kernels

constexpr int kListThreads = 256;
constexpr int kListRows = 4096;         // rows that a block of the listing kernel places at a time
constexpr int kListBlocks = 512;        // of the listing kernel at most

struct ListParams {
    const int64_t *target;      // cross entropy: a row takes part if its target is in 0 .. V - 1
    const int *entries;         // distillation: if it has entries
    int64_t V;
    int N, per_block;
    const char *x;
    int64_t x_stride;           // bytes
    int H;
    char *listed;               // the rows that take part, side by side
    int64_t listed_stride;      // bytes
    int *rows, *count;
    float *loss, *lse;          // forward: set to 0 for the other rows
    char *dx;                   // backward: the same
    int64_t dx_stride;
    const float *dloss;         // backward
    float *scale;               // backward: what g is scaled by (and its inverse)
    int f16;
    int copy;                   // copy the rows even if all take part
    float inv_t;
    Cut *cut;                   // backward: of dx's product, dw's, and dw's for the last piece
    int data_blocks, data_tile_m, data_k_tiles, data_slots;
    int weight_tiles, last_tiles, weight_slots;
    int parts;                  // of g
};

__device__ __forceinline__ bool takes_part(const ListParams &p, int i)
{
    return p.target ? uint64_t(p.target[i]) < uint64_t(p.V) : p.entries[i] > 0;
}

// Copies or clears a row of 16-bit values by one warp; 16 bytes at a time where
// both sides allow, four in flight.
__device__ __forceinline__ void warp_row(char *dst, const char *src, int H, int lane)
{
    const bool vec = (uintptr_t(dst) % 16) == 0 && (!src || uintptr_t(src) % 16 == 0);
    const int n = vec ? H / 8 : 0;
    for (int i = lane; i < n; i += 128) {
        uint4 v[4] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (src && i + 32 * j < n) v[j] = reinterpret_cast<const uint4 *>(src)[i + 32 * j];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + 32 * j < n) reinterpret_cast<uint4 *>(dst)[i + 32 * j] = v[j];
    }
    for (int i = n * 8 + lane; i < H; i += 32)
        reinterpret_cast<uint16_t *>(dst)[i] = src ? reinterpret_cast<const uint16_t *>(src)[i] : uint16_t(0);
}

// Lists the rows that take part, in order.  Each block counts the rows before
// its own by itself (a row is 8 bytes, from L2): one launch and no order among
// blocks, whose number is bounded so that the time grows with the rows and not with
// their square (33.5 million rows of 8, 2 tokens: forward 300 -> 56 ms).  Where every
// row takes part, nothing is copied.
__global__ void __launch_bounds__(kListThreads) list_kernel(const ListParams p)
{
    __shared__ int s_before, s_total, s_pos[kListRows];
    __shared__ unsigned int s_amax;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int first = blockIdx.x * p.per_block, last = first + min(p.per_block, p.N - first);
    if (tid == 0) {
        s_before = s_total = 0;
        s_amax = 0;
    }
    __syncthreads();
    int before = 0, total = 0;
    float amax = 0.0f;
    for (int i0 = tid; i0 < p.N; i0 += 8 * kListThreads) {       // eight loads in flight
        bool a[8];
        float d[8] = {};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * kListThreads;
            a[j] = i < p.N && takes_part(p, i);
            if (p.dloss && i < p.N) d[j] = p.dloss[i];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            total += a[j];
            before += a[j] && i0 + j * kListThreads < first;
            // a gradient that is not finite takes no part in the scale
            const float v = fabsf(d[j] * p.inv_t);
            if (a[j] && v < INFINITY) amax = fmaxf(amax, v);
        }
    }
    before = __reduce_add_sync(0xFFFFFFFFu, before);
    total = __reduce_add_sync(0xFFFFFFFFu, total);
    const unsigned int am = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(amax));    // amax >= 0: ordered as bits
    if (lane == 0) {
        atomicAdd(&s_before, before);
        atomicAdd(&s_total, total);
        atomicMax(&s_amax, am);
    }
    __syncthreads();
    total = s_total;
    if (blockIdx.x == 0 && tid == 0) {
        *p.count = total;
        if (p.scale) {
            // f16, which holds 2^-24 .. 2^16: the largest |dloss| / T goes to 2^13 (one below 2^-107
            // as high as 2^120 lifts it); bf16: to the next power of two, so that g stays where fp32 has it
            const float a = __uint_as_float(s_amax);
            float s = 1.0f, back = 1.0f;
            if (a > 0.0f && p.f16) {
                const float low = fmaxf(a, 0x1p-107f);
                s = 0x1p13f / low;
                back = low * 0x1p-13f;
            } else if (a > 0.0f) {
                int e;
                back = frexpf(a, &e);
                s = 1.0f / back;
            }
            p.scale[0] = s;
            p.scale[1] = back;
        }
    }
    if (blockIdx.x == 0 && warp == 1 && p.cut) {
        const Cut data = cut_of(max(1, (total + p.data_tile_m - 1) / p.data_tile_m) * p.data_blocks, p.data_k_tiles,
                                p.data_slots, lane);
        const int k_tiles = p.parts * max(1, (total + BK - 1) / BK);
        const Cut weight = cut_of(p.weight_tiles, k_tiles, p.weight_slots, lane);
        const Cut last = cut_of(p.last_tiles, k_tiles, p.weight_slots, lane);
        if (lane == 0) {
            p.cut[0] = data;
            p.cut[1] = weight;
            p.cut[2] = last;
        }
    }
    const bool side_by_side = total != p.N || p.copy;
    int pos = s_before;
    for (int from = first; from < last; from += kListRows) {
        const int to = min(last, from + kListRows);
        if (warp == 0) {
            for (int i = from; i < to; i += 32) {
                const bool a = i + lane < to && takes_part(p, i + lane);
                const unsigned int set = __ballot_sync(0xFFFFFFFFu, a);
                const int at = pos + __popc(set & ((1u << lane) - 1));
                if (a) p.rows[at] = i + lane;
                if (i + lane < to) s_pos[i + lane - from] = a ? at : -1;
                pos += __popc(set);
            }
        }
        if (!side_by_side) continue;
        __syncthreads();
        for (int i = from + warp; i < to; i += kListThreads / 32) {
            const int at = s_pos[i - from];
            if (at >= 0) {
                warp_row(p.listed + int64_t(at) * p.listed_stride, p.x + int64_t(i) * p.x_stride, p.H, lane);
            } else {
                if (p.dx) warp_row(p.dx + int64_t(i) * p.dx_stride, nullptr, p.H, lane);
                if (lane == 0 && p.loss) p.loss[i] = 0.0f;
                if (lane == 0 && p.lse) p.lse[i] = 0.0f;
            }
        }
        __syncthreads();            // the positions have been read
    }
    if (!side_by_side) return;
    // the last slice of rows of g^T x reads whole multiples of 64 rows
    const int end = min(p.N, max(BK, (total + BK - 1) / BK * BK));
    for (int i = total + blockIdx.x * (kListThreads / 32) + warp; i < end; i += gridDim.x * (kListThreads / 32))
        warp_row(p.listed + int64_t(i) * p.listed_stride, nullptr, p.H, lane);
}

struct TransposeParams {
    const char *x, *listed;
    int64_t x_stride, listed_stride;    // bytes
    const int *count;
    int N, H;
    char *out;
    int64_t out_stride;                 // bytes
};

constexpr int kTransTile = 64;

// x of the rows that take part, transposed: H rows of them, zeros up to a whole
// slice of K behind the last.  Tiles of 64 x 64 through shared memory, two rows
// of x to a 32-bit word of the result.
__global__ void __launch_bounds__(256) transpose_kernel(const TransposeParams p)
{
    __shared__ uint32_t s_tile[kTransTile][kTransTile / 2 + 1];     // [column][pair of rows]
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int count = *p.count, n0 = blockIdx.x * kTransTile;
    if (n0 >= max(1, count)) return;
    const char *src = count == p.N ? p.x : p.listed;
    const int64_t stride = count == p.N ? p.x_stride : p.listed_stride;
    const int pair = threadIdx.x >> 3, h = (threadIdx.x & 7) * 8;   // 32 pairs of rows, 8 columns each
    const int lane = threadIdx.x & 31;
    for (int h0 = blockIdx.y * kTransTile; h0 < p.H; h0 += gridDim.y * kTransTile) {
        uint16_t v[2][8];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int n = n0 + 2 * pair + r;
            const uint16_t *row = reinterpret_cast<const uint16_t *>(src + int64_t(n) * stride) + h0 + h;
            if (n < count && h0 + h + 8 <= p.H) {
                const uint4 w = *reinterpret_cast<const uint4 *>(row);
                memcpy(v[r], &w, 16);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[r][j] = n < count && h0 + h + j < p.H ? row[j] : uint16_t(0);
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) s_tile[h + j][pair] = uint32_t(v[0][j]) | uint32_t(v[1][j]) << 16;
        __syncthreads();
        // rows of the result have room for whole slices of 64
        for (int c = threadIdx.x >> 5; c < kTransTile && h0 + c < p.H; c += 8)
            reinterpret_cast<uint32_t *>(p.out + int64_t(h0 + c) * p.out_stride + int64_t(n0) * 2)[lane] = s_tile[c][lane];
    }
}

constexpr int kJoinThreads = 1024;

struct JoinParams {
    const float2 *part;
    int n_parts, N;
    const int *count, *rows;    // NULL: nothing was listed, every row is here
    const int64_t *target;
    int64_t V;
    const float *named;
    const float *share;         // distillation: [N][top] teacher's probabilities, in the order of the sorted tokens
    const int *order;           //               and where each stands in the caller's order
    const int *entries;
    const float *neg_entropy;   //               sum of p log p
    int top;
    float c1;
    float *loss, *lse, *top_logits;
};

// The tiles' maxima and sums of one row joined, and the loss formed from them.
//
// Cross entropy: s = sum over v != target of 2^(c1 z_v - m), r = c1 z_target - m and
// q = s 2^-r, what the other tokens have beside the target's 1.  The loss is
// log(1 + q): log1p of q where the target has more than half (it is then the
// maximum, r is 0 but for m's rounding, and the loss is never negative and as good
// as q, relatively), else ln 2 (log2(s + 2^r) - r), at least ln 2.  Relative to the
// loss that is what the terms are off by: a few roundings of 2^-24 of their
// distance from the maximum in log2 units, 2^-22 of each exponential, and the sum's.
//
// Distillation: sum_k p_k log p_k + ln 2 (log2 s - sum_k p_k (c1 z_k - m)), s over every
// token: off by some 2^-23 of the sizes of its terms whatever their sum is, so a
// student that is its teacher may see a loss of -1e-7.
template <int ROWS>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const JoinParams p)
{
    constexpr int kSlices = kJoinThreads / ROWS;        // of a row's parts, one a thread
    __shared__ float2 s_part[kSlices][ROWS];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int count = p.count ? *p.count : p.N;
    const int m0 = blockIdx.x * ROWS, m = m0 + threadIdx.x % ROWS;
    if (m0 >= count) return;
    const auto join = [](float2 a, float2 b) {
        const float hi = fmaxf(a.x, b.x), base = hi == -INFINITY ? 0.0f : hi;
        return make_float2(hi, a.y * exp2f(a.x - base) + b.y * exp2f(b.x - base));
    };
    // warp w joins row w; what its loss needs is on the way meanwhile
    const int r = warp, row = r < ROWS && m0 + r < count ? (count == p.N ? m0 + r : p.rows[m0 + r]) : -1;
    const int64_t target = p.target && row >= 0 ? p.target[row] : 0;
    const float named = p.target && row >= 0 ? p.named[m0 + r] : 0.0f;
    float2 mine = make_float2(-INFINITY, 0.0f);
    if (m < count)
#pragma unroll 4
        for (int b = threadIdx.x / ROWS; b < p.n_parts; b += kSlices) mine = join(mine, p.part[int64_t(b) * p.N + m]);
    s_part[threadIdx.x / ROWS][threadIdx.x % ROWS] = mine;
    __syncthreads();
    if (row < 0) return;
    float2 v = s_part[lane][r];
#pragma unroll
    for (int i = 32; i < kSlices; i += 32) v = join(v, s_part[lane + i][r]);
    float hi = v.x;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, d));
    const float base = hi == -INFINITY ? 0.0f : hi;
    float s = v.y * exp2f(v.x - base);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    if (p.target ? uint64_t(target) >= uint64_t(p.V) : p.entries[row] == 0) {   // takes no part
        if (lane == 0) p.loss[row] = p.lse[row] = 0.0f;
        return;
    }
    if (p.target) {
        if (lane == 0) {
            const float at = fmaf(named, p.c1, -base);
            const float q = s * exp2f(-at), l2 = log2f(s + exp2f(at));
            p.loss[row] = q < 1.0f ? log1pf(q) : kLn2 * (l2 - at);
            p.lse[row] = kLn2 * (base + l2);
        }
        return;
    }
    const float l2 = log2f(s);
    const int n = p.entries[row];
    const int64_t at = int64_t(row) * p.top;
    float mean = 0.0f;          // sum of p_k (c1 z_k - m)
    for (int e = lane; e < n; e += 32) {
        const float z = p.named[at + e], share = p.share[at + e];
        // a share of 0 has no part in the sum
        if (share != 0.0f) mean = fmaf(share, fmaf(z, p.c1, -base), mean);
        p.top_logits[at + p.order[at + e]] = z;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mean += __shfl_xor_sync(0xFFFFFFFFu, mean, d);
    if (lane == 0) {
        p.loss[row] = p.neg_entropy[row] + kLn2 * (l2 - mean);
        p.lse[row] = kLn2 * (base + l2);
    }
}

struct TeacherParams {
    const int64_t *index;
    const char *logit;
    int64_t index_stride, logit_stride;     // elements
    int dtype;
    int64_t V;
    int top, pow2;
    float inv_t;
    int *sorted, *order, *entries;
    float *share, *neg_entropy;
    float *top_logits;          // forward: set to 0 where there is no entry
};

__device__ __forceinline__ float teacher_logit(const TeacherParams &p, int64_t i)
{
    const char *at = p.logit + i * (p.dtype == GLU_F32 ? 4 : 2);
    return p.dtype == GLU_F32 ? Codec<float>::load1(at)
                              : p.dtype == GLU_F16 ? Codec<__half>::load1(at) : Codec<__nv_bfloat16>::load1(at);
}

__device__ __forceinline__ float block_reduce(float v, bool maximum, float *s_red)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float o = __shfl_xor_sync(0xFFFFFFFFu, v, d);
        v = maximum ? fmaxf(v, o) : v + o;
    }
    __syncthreads();            // the last call's values have been read
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s_red[0];
    for (int w = 1; w < int(blockDim.x >> 5); ++w) v = maximum ? fmaxf(v, s_red[w]) : v + s_red[w];
    return v;
}

// One row of the teacher's entries a block: sorted by token (a bitonic network in
// shared memory; entries of one token stay in their order), the softmax of their
// logits at T, and the sum of p log p.  An entry whose token is outside the
// vocabulary or whose logit is -inf is none.
__global__ void __launch_bounds__(512) teacher_kernel(const TeacherParams p)
{
    extern __shared__ uint64_t s_key[];             // token << 32 | place in the caller's order
    __shared__ float s_red[16];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row = blockIdx.x;
    const int64_t *index = p.index + row * p.index_stride;
    float hi = -INFINITY;
    int n = 0, any_nan = 0;
    for (int k = threadIdx.x; k < p.pow2; k += blockDim.x) {
        uint64_t key = uint64_t(INT32_MAX) << 32 | uint32_t(k);
        if (k < p.top) {
            const int64_t v = index[k];
            const float t = teacher_logit(p, row * p.logit_stride + k);
            if (uint64_t(v) < uint64_t(p.V) && t != -INFINITY) {
                key = uint64_t(v) << 32 | uint32_t(k);
                any_nan |= t != t;
                hi = fmaxf(hi, t);
                ++n;
            } else if (p.top_logits) {
                p.top_logits[row * p.top + k] = 0.0f;
            }
        }
        s_key[k] = key;
    }
    hi = block_reduce(hi, true, s_red);
    n = int(block_reduce(float(n), false, s_red));
    any_nan = __syncthreads_or(any_nan);
    if (any_nan) hi = NAN;
    for (int size = 2; size <= p.pow2; size <<= 1) {
        for (int step = size >> 1; step > 0; step >>= 1) {
            __syncthreads();
            for (int i = threadIdx.x; i < p.pow2 / 2; i += blockDim.x) {
                const int a = 2 * i - (i & (step - 1)), b = a + step;
                const uint64_t ka = s_key[a], kb = s_key[b];
                if ((ka > kb) == ((a & size) == 0)) {
                    s_key[a] = kb;
                    s_key[b] = ka;
                }
            }
        }
    }
    __syncthreads();
    // the sorted entries' shares; (t - hi) before / T: a lowest logit does not overflow
    float sum = 0.0f;
    for (int e = threadIdx.x; e < n; e += blockDim.x) {
        const int k = int(uint32_t(s_key[e]));
        sum += expf((teacher_logit(p, row * p.logit_stride + k) - hi) * p.inv_t);
    }
    sum = block_reduce(sum, false, s_red);
    const float log_sum = logf(sum), inv = 1.0f / sum;
    float ent = 0.0f;
    for (int e = threadIdx.x; e < p.top; e += blockDim.x) {
        const int64_t at = row * p.top + e;
        const uint64_t key = s_key[e];
        const int k = int(uint32_t(key));
        p.sorted[at] = e < n ? int(key >> 32) : INT32_MAX;
        p.order[at] = k;
        if (e < n) {
            const float d = (teacher_logit(p, row * p.logit_stride + k) - hi) * p.inv_t;
            const float share = expf(d) * inv;
            p.share[at] = share;
            if (share != 0.0f) ent = fmaf(share, d - log_sum, ent);
        }
    }
    ent = block_reduce(ent, false, s_red);
    if (threadIdx.x == 0) {
        p.entries[row] = n;
        p.neg_entropy[row] = ent;
    }
}

struct NamedParams {
    const int *count, *rows, *sorted, *order, *entries;
    const float *share, *top_logits, *lse, *dloss, *scale;
    int N, top;
    int64_t first, cols;        // the piece of the vocabulary
    float c1, inv_t;
    char *g;
    int64_t g_stride;           // bytes
    int parts;                  // of g, the second part_cols columns behind the first
    int64_t part_cols;
};

// Distillation: the entries of g that the teacher names, formed anew from the
// forward pass's logits (g as stored is rounded: the share could not be taken off
// it).  One block a row; the first of a token's entries sums its shares.
template <class T>
__global__ void __launch_bounds__(128) named_grad_kernel(const NamedParams p)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int count = *p.count, m = blockIdx.x;
    if (m >= count) return;
    const int row = count == p.N ? m : p.rows[m];
    const int n = p.entries[row];
    const int64_t at = int64_t(row) * p.top;
    const float coef = p.dloss[row] * p.inv_t * p.scale[0];
    if (coef == 0.0f) return;
    const float shift = -p.lse[row] * kLog2e;
    for (int e = threadIdx.x; e < n; e += blockDim.x) {
        const int v = p.sorted[at + e];
        if (v < p.first || v >= p.first + p.cols || (e > 0 && p.sorted[at + e - 1] == v)) continue;
        float share = p.share[at + e];
        for (int i = e + 1; i < n && p.sorted[at + i] == v; ++i) share += p.share[at + i];
        const float z = p.top_logits[at + p.order[at + e]];
        const float f = coef * (exp2_fast(fmaf(z, p.c1, shift)) - share);
        char *dst = p.g + int64_t(m) * p.g_stride + (v - p.first) * 2;
        Codec<T>::store1(dst, f);
        if (p.parts == 2) Codec<T>::store1(dst + p.part_cols * 2, f - Codec<T>::load1(dst));
    }
}

struct SumParams {
    const float *tail;          // parts of tile_m x tile_n sums
    const float *sums;          // several pieces: the sums of the tiles that were not cut
    int64_t ld;                 // floats
    const int *count, *rows;
    int weight;                 // the rows are tokens, K the listed rows (else the other way round)
    int N, cols, m_rows, n_blocks, group_m, tile_m, tile_n;
    const Cut *cut;
    const float *scale;
    char *out;
    int64_t out_stride;         // bytes
};

// The tiles kept as fp32 sums, rounded once: their parts added in order.
template <class T>
__global__ void __launch_bounds__(256) sum_kernel(const SumParams p)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int count = *p.count;
    const int m_rows = p.weight ? p.m_rows : count;
    const int m_blocks = max(1, (m_rows + p.tile_m - 1) / p.tile_m);
    const int n_tiles = m_blocks * p.n_blocks;
    const Cut cut = *p.cut;
    const int tail = n_tiles - cut.whole;
    const float unscale = p.scale[1];
    const bool vec = (uintptr_t(p.out) % 8) == 0 && p.out_stride % 8 == 0;
    const int quads = p.tile_n / 4, per_tile = p.tile_m * quads;
    const int first = p.sums ? 0 : cut.whole;
    const int64_t n = int64_t(n_tiles - first) * per_tile;
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) {
        const int t = first + int(i / per_tile), j = int(i % per_tile);
        const Tile o = tile_of(p.group_m, p.n_blocks, t, m_blocks);
        const int r = j / quads, x = j % quads * 4;
        const int m = o.mb * p.tile_m + r, c = o.nb * p.tile_n + x;
        if (m >= m_rows || c >= p.cols) continue;
        float4 a;
        if (t < cut.whole) {
            a = *reinterpret_cast<const float4 *>(p.sums + int64_t(m) * p.ld + c);
        } else {
            const float *src = p.tail + (int64_t(t - cut.whole) * p.tile_m + r) * p.tile_n + x;
            const int64_t step = int64_t(tail) * p.tile_m * p.tile_n;
            a = *reinterpret_cast<const float4 *>(src);
#pragma unroll 4
            for (int s = 1; s < cut.parts; ++s) {
                const float4 b = *reinterpret_cast<const float4 *>(src + s * step);
                a.x += b.x;
                a.y += b.y;
                a.z += b.z;
                a.w += b.w;
            }
        }
        const int row = !p.weight && count != p.N ? p.rows[m] : m;
        char *dst = p.out + int64_t(row) * p.out_stride + int64_t(c) * 2;
        const float f[4] = {a.x * unscale, a.y * unscale, a.z * unscale, a.w * unscale};
        if (vec && c + 4 <= p.cols) {
            *reinterpret_cast<uint2 *>(dst) = make_uint2(Codec<T>::put(f), Codec<T>::put(f + 2));
        } else {
            for (int e = 0; e < 4 && c + e < p.cols; ++e) Codec<T>::store1(dst + 2 * e, f[e]);
        }
    }
}

}  // namespace loss
}  // namespace glu

// ---------------------------------------------------------------- host side

namespace glu {
namespace loss {

cudaError_t timeouts(unsigned int *count, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(count, g_loss_timeouts, sizeof(unsigned int));
    if (e == cudaSuccess && reset) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_loss_timeouts, &zero, sizeof(unsigned int));
    }
    return e;
}

namespace {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxSize = INT32_MAX - 65536;
constexpr int kMaxTop = 1024;
// g of one piece of the vocabulary, or 256 tokens of it where those are more; a smaller
// workspace takes smaller pieces
constexpr uint64_t kPieceBytes = uint64_t(1) << 30;
constexpr int64_t kMinPiece = 256;

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

bool make_map(CUtensorMap *m, CUtensorMapDataType type, const void *base, int64_t rows, int64_t cols,
              int64_t stride_bytes, int box_cols, int box_rows, CUtensorMapSwizzle swizzle)
{
    EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(stride_bytes)};
    const cuuint32_t box[2] = {cuuint32_t(box_cols), cuuint32_t(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, type, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

using GemmFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, Params);

struct Variant {
    GemmFn fn;
    int smem, bn, ctas, id, mode;
};

constexpr int kVariants = 22;

template <int MODE, int BN, int CTAS>
Variant variant(bool bf16, int id)
{
    return {bf16 ? loss_gemm_kernel<MODE, __nv_bfloat16, BN, CTAS> : loss_gemm_kernel<MODE, __half, BN, CTAS>,
            Shape<MODE, BN, CTAS>::kSmemBytes, BN, CTAS, id, MODE};
}

// Blocks (or pairs) of a variant that fit on the device at once, and the
// shared-memory opt-in, once per device.
std::atomic<int> g_slots[kMaxDevices][2][kVariants];

int slots_of(const Variant &v, bool bf16, int dev, int sms, int *out)
{
    std::atomic<int> &slots = g_slots[dev % kMaxDevices][bf16][v.id];
    int n = slots.load(std::memory_order_acquire);
    if (n == 0) {
        // the warps' register split draws on what the kernel is launched with
        cudaFuncAttributes fa{};
        cudaError_t e = cudaFuncGetAttributes(&fa, reinterpret_cast<const void *>(v.fn));
        if (e == cudaSuccess && fa.numRegs < kRegsLaunch) e = cudaErrorInvalidKernelImage;
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(reinterpret_cast<const void *>(v.fn), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     v.smem);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return glu::cuda_fail(e);
        }
        n = sms;
        if (v.ctas > 1) {
            cudaLaunchConfig_t q{};
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = unsigned(v.ctas);
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            q.blockDim = dim3(kThreads);
            q.dynamicSmemBytes = size_t(v.smem);
            q.gridDim = dim3(unsigned(sms - sms % v.ctas));
            q.attrs = attr;
            q.numAttrs = 1;
            int clusters = 0;
            e = cudaOccupancyMaxActiveClusters(&clusters, reinterpret_cast<const void *>(v.fn), &q);
            if (e != cudaSuccess || clusters <= 0) {
                (void)cudaGetLastError();
                clusters = sms / v.ctas;
            }
            n = clusters;
        }
        slots.store(n, std::memory_order_release);
    }
    *out = n;
    return GLU_OK;
}

// A launch that may overlap the tail of the one before it in the stream (every
// kernel here waits for that grid before it touches memory).
int launch(const void *fn, dim3 grid, unsigned threads, size_t smem, unsigned cluster, void **args, cudaStream_t s)
{
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
    if (e != cudaSuccess) {     // retry without the dependent-launch attribute
        (void)cudaGetLastError();
        cfg.numAttrs = 1;
        e = cudaLaunchKernelExC(&cfg, fn, args);
    }
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return glu::cuda_fail(e);
    }
    return GLU_OK;
}

int device(int *dev, int *sms)
{
    cudaError_t e = cudaGetDevice(dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return glu::cuda_fail(e);
    }
    return GLU_OK;
}

// Everything a pass gets; what it does not use stays empty.
struct Call {
    const void *x;
    int64_t x_stride;
    const void *w;
    int64_t w_stride;
    int64_t N, H, V;
    int dtype;
    const int64_t *target;      // cross entropy
    const int64_t *index;       // distillation
    int64_t index_stride;
    const void *logit;
    int64_t logit_stride;
    int64_t top;
    int logit_dtype;
    float temperature;
    float *loss, *lse, *top_logits;
    const float *dloss;
    void *dx;
    int64_t dx_stride;
    void *dw;
    int64_t dw_stride;
    void *workspace;
    size_t workspace_bytes;
    bool backward, distill;
};

constexpr int kSms = 152;              // what the parts of K are counted for

// How a pass divides its work and its workspace (offsets in bytes).
struct Plan {
    int64_t piece;              // backward: tokens of a piece
    int pieces;
    int ctas, bn;               // of the logits' product: blocks a tile, half its columns
    int64_t tail_rows[2];       // rows of the parts of tiles that are kept apart: of dx, of dw
    int64_t ld;                 // of the sums over pieces, in floats
    bool lists;                 // the rows that take part are listed: not for a forward pass over one block of rows
    bool transpose;             // x transposed for dw
    bool copy;                  // x's rows copied whether or not all take part
    int parts;                  // 16-bit parts of g
    int64_t part_cols;          // columns of one
    int64_t g_stride, listed_stride, xt_stride;     // bytes
    uint64_t rows, listed, part, named, sorted, order, entries, share, entropy, g, xt, tail[2], sums, bytes;
};

// Column-tile width of the logits' product: the fewest rows of x and w moved,
// counted in rounds of tiles over the GPU (the widest on a tie).  Tiles of 64 columns
// only for one block of rows: they fill the GPU with the smallest calls (dx of 16 x
// 1024, 8192 tokens 25.3 -> 23.5 us).
int pick_bn(int64_t m_blocks, int64_t V, int64_t slots, int64_t a_rows, bool one_block)
{
    int best = 128;
    int64_t best_cost = -1;
    for (int bn : {128, 96, 64, 32}) {
        if (bn == 32 && !one_block) break;
        const int64_t tiles = m_blocks * ((V + 2 * bn - 1) / (2 * bn));
        const int64_t cost = (tiles + slots - 1) / slots * (a_rows + 2 * bn);
        if (best_cost < 0 || cost < best_cost) {
            best = bn;
            best_cost = cost;
        }
    }
    return best;
}

// dw's product reads g as an MN-major operand, and x too unless it is transposed
// first.  With x K-major the tensor cores wait less for shared memory (busy 72 % of
// the cycles with both operands MN-major, 81 % with one), which saves some 4 % of the
// product, 4.5e-11 N H V us; transposing takes a launch, about 1.1 us behind the
// others, and moves x twice, 4.2e-7 N H us.  So it pays where N H (V - 9400) is above
// 2.5e10.  Measured, g and dw together, without -> with: 4096 x 4096, 65536 tokens
// 2389 -> 2340 us, 16384 641 -> 634, 8192 336 -> 339; 2048 x 2048, 32000 343 -> 339,
// 16384 182 -> 180, 8192 110 -> 111; 512 x 4096, 32000 209 -> 207, 16384 120 -> 121;
// 512 x 1024, 65536 120.4 -> 119.8, 32000 74.6 -> 74.9.  Up to 128 rows dw's bytes bound
// the product: 256 x 4096, 65536 257 -> 250, 128 x 4096, 65536 200 -> 203.
bool transposes(int64_t N, int64_t H, int64_t V)
{
    return N > BM && double(N) * double(H) * double(V - 9400) > 2.5e10;
}

// Half the columns of a gradient product's tile: 128 columns where a tile of 256 would
// be half empty.
int grad_bn(int64_t H) { return H <= 128 ? 64 : 128; }

// 16-bit parts of g.  One rounds g to the inputs' type.  With a second for what the
// first leaves, g has 16 bits (f16: 22) and dx and dw are off by no more than their own
// rounding (16 x 1024, 8192 tokens, 8 teacher's entries, against 64 bits in the 2-norm:
// 2.4e-3 -> 1.7e-3), at twice the tensor cores' work.  Up to 64 rows that hides behind
// w's and dw's bytes: step of 64 x 4096, 32768 tokens 216 -> 225 us, 16 x 1024, 8192
// 45.7 -> 47.7, 64 x 1000, 50001 117 -> 125.  With more rows it does not: 96 x 4096,
// 32768 221 -> 247, 256 x 4096 260 -> 332, 1024 x 4096 670 -> 978, 4096 x 4096, 131072
// 9250 -> 13970; there one part is the choice, as in training with 16-bit logits (4096 x
// 4096, 131072: off 1.82e-3 of 64 bits, 1.66e-3 of it dx's own rounding; with 64
// teacher's entries a row 2.3e-3).
int g_parts(int64_t N) { return N <= BM / 2 ? 2 : 1; }

Plan make_plan(const Call &c, int64_t piece)
{
    Plan p{};
    uint64_t at = 0;
    const auto take = [&](uint64_t bytes) {
        const uint64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const uint64_t N = uint64_t(c.N), top = uint64_t(c.top);
    // where x's rows are off 32 bytes the copy engine reads a sector more for every
    // 128 bytes: such x is copied as if rows were missing (rows of 2064 bytes, 777 x
    // 1030, 30001 tokens: backward 190 -> 185 us; of 4000 bytes, 333 x 1999, 50001,
    // it would take 290 for 286)
    p.copy = c.N > BM && c.x_stride % 16 != 0;
    p.lists = c.backward || c.N > BM;   // where it is not, rows without a token cost nothing
    p.listed_stride = round_up(c.H, 64) * 2;
    if (p.lists) {
        p.rows = take(4 * N + 64);      // the count, the scale and its inverse, the cuts, then the list (from byte 64)
        p.listed = take(N * uint64_t(p.listed_stride));
    }
    if (c.distill) {
        p.sorted = take(4 * N * top);
        p.order = take(4 * N * top);
        p.share = take(4 * N * top);
        p.entries = take(4 * N);
        p.entropy = take(4 * N);
    }
    // sized for the whole GPU whatever the device, so that the bytes asked for hold
    p.ctas = c.N > BM ? 2 : 1;
    const int64_t tile_m = BM * p.ctas, m_blocks = (c.N + tile_m - 1) / tile_m;
    p.bn = pick_bn(m_blocks, c.backward ? piece : c.V, kSms / p.ctas, p.ctas == 1 ? round_up(c.N, 8) : tile_m,
                   p.ctas == 1);
    if (!c.backward) {
        // two halves of a tile, each joined by itself
        p.part = take(16 * N * uint64_t((c.V + 2 * p.bn - 1) / (2 * p.bn)));
        p.named = take(4 * N * (c.distill ? top : 1));
    } else {
        p.piece = piece;
        p.pieces = int((c.V + piece - 1) / piece);
        p.parts = g_parts(c.N);
        p.part_cols = round_up(piece, 64);
        p.g_stride = p.parts * p.part_cols * 2;
        p.g = take(N * uint64_t(p.g_stride));
        p.transpose = c.dw && transposes(c.N, c.H, c.V);
        p.xt_stride = round_up(c.N, 64) * 2;
        if (p.transpose) p.xt = take(uint64_t(c.H) * uint64_t(p.xt_stride));
        // The parts of the tiles that are cut, whatever number of rows takes part.  Those of
        // dx add up over the pieces, with dw's in between: each has its own.
        const int64_t tile_n = grad_bn(c.H) * 2, n_blocks = (c.H + tile_n - 1) / tile_n;
        const auto room = [&](int64_t tiles, int64_t k_tiles, int64_t slots) {
            const int64_t cuts = k_tiles / 4 < kMaxParts ? k_tiles / 4 : kMaxParts;     // of one tile at most
            const int64_t most = tiles * cuts < kTailRounds * slots ? tiles * cuts : kTailRounds * slots;
            return cuts < 2 ? int64_t(0) : most;
        };
        p.tail_rows[0] = c.dx ? room(m_blocks * n_blocks, (piece + BK - 1) / BK, kSms / p.ctas) * tile_m : 0;
        p.tail_rows[1] =
            c.dw ? room((piece + 255) / 256 * n_blocks, p.parts * ((c.N + BK - 1) / BK), kSms / 2) * 256 : 0;
        for (int i = 0; i < 2; ++i) p.tail[i] = take(4 * uint64_t(p.tail_rows[i]) * uint64_t(tile_n));
        p.ld = round_up(c.H, 4);
        if (c.dx && p.pieces > 1) p.sums = take(4 * N * uint64_t(p.ld));
    }
    p.bytes = at;
    return p;
}

// Pieces of at most kPieceBytes of g, about equal, whole tiles.
int64_t default_piece(int64_t N, int64_t V)
{
    int64_t most = int64_t(kPieceBytes / (2 * uint64_t(g_parts(N)) * uint64_t(N))) / kMinPiece * kMinPiece;
    if (most < kMinPiece) most = kMinPiece;
    const int64_t pieces = (V + most - 1) / most;
    return round_up((V + pieces - 1) / pieces, kMinPiece) < V ? round_up((V + pieces - 1) / pieces, kMinPiece) : V;
}

bool plan_for(const Call &c, uint64_t bytes, Plan *out)
{
    int64_t piece = c.backward ? default_piece(c.N, c.V) : c.V;
    while (true) {
        *out = make_plan(c, piece);
        if (out->bytes <= bytes) return true;
        if (!c.backward || piece <= kMinPiece) return false;
        piece = round_up((piece + 1) / 2, kMinPiece) < piece ? round_up((piece + 1) / 2, kMinPiece) : piece - kMinPiece;
        if (piece < kMinPiece) piece = kMinPiece;
    }
}

// Argument rules of the four entry points; no CUDA call.
int validate(Call &c, bool *empty)
{
    *empty = false;
    if (c.dtype != GLU_F16 && c.dtype != GLU_BF16) return GLU_ERR_ENUM;
    if (c.distill && c.logit_dtype != GLU_F32 && c.logit_dtype != GLU_F16 && c.logit_dtype != GLU_BF16)
        return GLU_ERR_ENUM;
    if (c.N < 0 || c.H < 1 || c.V < 1 || c.N > kMaxSize || c.H > kMaxSize || c.V > kMaxSize) return GLU_ERR_SHAPE;
    if (c.distill && (c.top < 1 || c.top > kMaxTop)) return GLU_ERR_SHAPE;
    if (c.distill && !(c.temperature >= 0x1p-10f && c.temperature <= 0x1p10f)) return GLU_ERR_VALUE;
    if (c.backward && !c.dx && !c.dw) {
        *empty = true;
        return GLU_OK;
    }
    if (c.N == 0) {             // dw is 0, nothing else is left to do
        *empty = true;
        if (c.V == 1) c.dw_stride = c.H;    // separates nothing
        if (c.backward && c.dw && c.dw_stride < c.H) return GLU_ERR_STRIDE;
        if (uintptr_t(c.dw) % 2) return GLU_ERR_STRIDE;
        return GLU_OK;
    }
    if (!c.x || !c.w || !c.lse || !c.workspace || (!c.distill && !c.target) ||
        (c.distill && (!c.index || !c.logit || !c.top_logits)) || ((!c.backward || !c.distill) && !c.loss) ||
        (c.backward && !c.dloss))
        return GLU_ERR_NULL;
    // strides that separate nothing
    if (c.N == 1) {
        c.x_stride = round_up(c.H, 8);
        c.dx_stride = c.H;
        c.index_stride = c.logit_stride = c.top;
    }
    if (c.V == 1) {
        c.w_stride = round_up(c.H, 8);
        c.dw_stride = c.H;
    }
    if (c.x_stride < c.H || c.w_stride < c.H || (c.dx && c.dx_stride < c.H) || (c.dw && c.dw_stride < c.H) ||
        (c.distill && (c.index_stride < c.top || c.logit_stride < c.top)))
        return GLU_ERR_STRIDE;
    // the tensor-memory accelerator: 16-byte aligned bases and strides (below 2^40 bytes)
    if (uintptr_t(c.x) % 16 || uintptr_t(c.w) % 16 || c.x_stride % 8 || c.w_stride % 8 ||
        c.x_stride >= (int64_t(1) << 39) || c.w_stride >= (int64_t(1) << 39))
        return GLU_ERR_STRIDE;
    if (uintptr_t(c.target) % 8 || uintptr_t(c.index) % 8 || uintptr_t(c.loss) % 4 || uintptr_t(c.lse) % 4 ||
        uintptr_t(c.top_logits) % 4 || uintptr_t(c.dloss) % 4 || uintptr_t(c.dx) % 2 || uintptr_t(c.dw) % 2 ||
        uintptr_t(c.logit) % (c.logit_dtype == GLU_F32 ? 4 : 2) || uintptr_t(c.workspace) % 256)
        return GLU_ERR_STRIDE;
    // 0 .. 4 read only, the rest outputs and the workspace
    enum { X, W, Names, Logit, Dloss, Loss, Lse, Top, Dx, Dw, Work, kSpans };
    Span s[kSpans] = {};
    const int64_t top = c.distill ? c.top : 0;
    bool fits = span(c.x, c.N, c.x_stride, c.H, 2, &s[X]) && span(c.w, c.V, c.w_stride, c.H, 2, &s[W]) &&
                span(c.loss, c.loss ? 1 : 0, 0, c.N, 4, &s[Loss]) && span(c.lse, 1, 0, c.N, 4, &s[Lse]) &&
                span(c.dloss, c.backward ? 1 : 0, 0, c.N, 4, &s[Dloss]) &&
                span(c.dx, c.dx ? c.N : 0, c.dx_stride, c.H, 2, &s[Dx]) &&
                span(c.dw, c.dw ? c.V : 0, c.dw_stride, c.H, 2, &s[Dw]) &&
                (c.distill ? span(c.index, c.N, c.index_stride, top, 8, &s[Names]) &&
                                 span(c.logit, c.N, c.logit_stride, top, c.logit_dtype == GLU_F32 ? 4 : 2, &s[Logit]) &&
                                 span(c.top_logits, c.N, top, top, 4, &s[Top])
                           : span(c.target, 1, 0, c.N, 8, &s[Names]));
    s[Work].lo = uintptr_t(c.workspace);
    fits = fits && !__builtin_add_overflow(s[Work].lo, uint64_t(c.workspace_bytes), &s[Work].hi);
    if (!fits) return GLU_ERR_SHAPE;
    for (int o = c.backward ? int(Dx) : int(Loss); o < kSpans; ++o)
        for (int i = 0; i < o; ++i)
            if (overlap(s[o], s[i])) return GLU_ERR_ALIAS;
    return GLU_OK;
}

// The operands of the tensor-memory accelerator are in the current device's memory.
int check_device(const Call &c, int dev)
{
    for (const void *q : {c.x, c.w, static_cast<const void *>(c.workspace), static_cast<const void *>(c.dx),
                          static_cast<const void *>(c.dw)}) {
        if (!q) continue;
        cudaPointerAttributes at{};
        const cudaError_t e = cudaPointerGetAttributes(&at, q);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return glu::cuda_fail(e);
        }
        if (at.type != cudaMemoryTypeDevice || at.device != dev) return GLU_ERR_VALUE;
    }
    return GLU_OK;
}

struct Run {
    const Call &c;
    const Plan &plan;
    cudaStream_t s;
    int dev, sms;
    bool bf16;
    char *ws;
    CUtensorMapDataType type16;

    int *count() const { return reinterpret_cast<int *>(ws + plan.rows); }
    float *scale() const { return reinterpret_cast<float *>(ws + plan.rows + 8); }
    Cut *cuts() const { return reinterpret_cast<Cut *>(ws + plan.rows + 16); }
    int *rows() const { return reinterpret_cast<int *>(ws + plan.rows + 64); }
    template <class P>
    P *at(uint64_t offset) const { return reinterpret_cast<P *>(ws + offset); }
    float inv_t() const { return c.distill ? 1.0f / c.temperature : 1.0f; }
    float c1() const { return c.distill ? float(1.4426950408889634 / double(c.temperature)) : kLog2e; }

    int teacher() const
    {
        TeacherParams t{};
        t.index = c.index;
        t.index_stride = c.index_stride;
        t.logit = static_cast<const char *>(c.logit);
        t.logit_stride = c.logit_stride;
        t.dtype = c.logit_dtype;
        t.V = c.V;
        t.top = int(c.top);
        t.pow2 = 2;
        while (t.pow2 < t.top) t.pow2 *= 2;
        t.inv_t = inv_t();
        t.sorted = at<int>(plan.sorted);
        t.order = at<int>(plan.order);
        t.share = at<float>(plan.share);
        t.entries = at<int>(plan.entries);
        t.neg_entropy = at<float>(plan.entropy);
        t.top_logits = c.backward ? nullptr : c.top_logits;
        void *args[] = {&t};
        const unsigned threads = unsigned(t.pow2 / 2 < 32 ? 32 : t.pow2 / 2);
        return launch(reinterpret_cast<const void *>(&teacher_kernel), unsigned(c.N), threads, size_t(t.pow2) * 8, 1,
                      args, s);
    }

    int list() const
    {
        ListParams l{};
        l.target = c.distill ? nullptr : c.target;
        l.entries = c.distill ? at<int>(plan.entries) : nullptr;
        l.V = c.V;
        l.N = int(c.N);
        l.per_block = int((c.N + kListBlocks - 1) / kListBlocks);
        if (l.per_block < 16) l.per_block = 16;
        l.x = static_cast<const char *>(c.x);
        l.x_stride = c.x_stride * 2;
        l.H = int(c.H);
        l.listed = at<char>(plan.listed);
        l.listed_stride = plan.listed_stride;
        l.rows = rows();
        l.count = count();
        l.inv_t = inv_t();
        l.copy = plan.copy;
        if (c.backward) {
            l.dx = static_cast<char *>(c.dx);
            l.dx_stride = c.dx_stride * 2;
            l.dloss = c.dloss;
            l.scale = scale();
            l.f16 = !bf16;
            const int64_t n_blocks = (c.H + 2 * grad_bn(c.H) - 1) / (2 * grad_bn(c.H));
            l.cut = cuts();
            l.data_blocks = int(n_blocks);
            l.data_tile_m = BM * plan.ctas;
            l.parts = plan.parts;
            l.data_k_tiles = int((plan.piece + BK - 1) / BK);
            l.data_slots = kSms / plan.ctas;
            l.weight_tiles = int((plan.piece + 255) / 256 * n_blocks);
            l.last_tiles = int((c.V - (plan.pieces - 1) * plan.piece + 255) / 256 * n_blocks);
            l.weight_slots = kSms / 2;
        } else {
            l.loss = c.loss;
            l.lse = c.lse;
        }
        void *args[] = {&l};
        return launch(reinterpret_cast<const void *>(&list_kernel), unsigned((c.N + l.per_block - 1) / l.per_block),
                      kListThreads, 0, 1, args, s);
    }

    bool map16(CUtensorMap *m, const void *base, int64_t r, int64_t cols, int64_t stride_bytes, int box_cols,
               int box_rows, CUtensorMapSwizzle sw) const
    {
        return make_map(m, type16, base, r, cols, stride_bytes, box_cols, box_rows, sw);
    }

    // One product, its grid sized for all rows.
    int product(const Variant &v, CUtensorMap &a, CUtensorMap &b, CUtensorMap &listed, CUtensorMap &out,
                CUtensorMap &tail, Params &p, int64_t all_rows, int64_t row_bytes, glu_launch_info_t *info) const
    {
        int n_slots = 0;
        if (int st = slots_of(v, bf16, dev, sms, &n_slots)) return st;
        const int64_t tile_m = int64_t(BM) * v.ctas;
        const int64_t m_blocks = (all_rows + tile_m - 1) / tile_m;
        p.count = plan.lists ? count() : nullptr;
        p.rows = rows();
        p.N = int(c.N);
        p.copied = plan.copy && plan.lists;
        p.n_blocks = int((p.cols + 2 * v.bn - 1) / (2 * v.bn));
        // row blocks per group: their rows of A (about 48 MiB) stay in L2 while B
        // streams past once; where one block row is more than that, tiles that run
        // side by side form a square
        int64_t group = (int64_t(48) << 20) / (tile_m * row_bytes);
        if (group < 8) group = 8;
        // dw: g, which is read once, makes way for x, which is read for every row block: a
        // round of tiles takes every column of a few row blocks (1024 x 4096, 32768 tokens:
        // dw's product 0.8 % faster, 4096 x 4096, 131072: 0.4 %)
        if (is_weight(v.mode)) group = (kSms / v.ctas + p.n_blocks - 1) / p.n_blocks;
        p.group_m = int(group > m_blocks ? m_blocks : group);
        const int64_t tiles = m_blocks * p.n_blocks;
        if (tiles + kTailRounds * kSms > INT32_MAX / 2) return GLU_ERR_SHAPE;
        // the gradients' tiles may be cut into up to kMaxParts parts
        const int64_t items = is_gradient(v.mode) ? tiles * kMaxParts : tiles;
        const int64_t clusters = items < n_slots ? items : n_slots;
        void *args[] = {&a, &b, &listed, &out, &tail, &p};
        if (int st = launch(reinterpret_cast<const void *>(v.fn), unsigned(clusters * v.ctas), kThreads,
                            size_t(v.smem), unsigned(v.ctas), args, s))
            return st;
        info->launched = 1;
        info->unroll = v.ctas;
        info->threads = kThreads;
        info->grid = int32_t(clusters * v.ctas);
        info->vector_units = tiles;
        return GLU_OK;
    }

    // The logits' product over tokens first .. first + cols.
    int logits(bool grad, int64_t first, int64_t cols, glu_launch_info_t *info) const
    {
        const int ctas = plan.ctas, bn = plan.bn;
        Variant v{};
        if (!grad)
            v = ctas == 1 ? (bn == 32   ? variant<kStats, 32, 1>(bf16, 18)
                             : bn == 64 ? variant<kStats, 64, 1>(bf16, 0)
                             : bn == 96 ? variant<kStats, 96, 1>(bf16, 1)
                                        : variant<kStats, 128, 1>(bf16, 2))
                          : (bn == 64   ? variant<kStats, 64, 2>(bf16, 3)
                             : bn == 96 ? variant<kStats, 96, 2>(bf16, 4)
                                        : variant<kStats, 128, 2>(bf16, 5));
        else
            v = ctas == 1 ? (bn == 32   ? variant<kGrad, 32, 1>(bf16, 19)
                             : bn == 64 ? variant<kGrad, 64, 1>(bf16, 6)
                             : bn == 96 ? variant<kGrad, 96, 1>(bf16, 7)
                                        : variant<kGrad, 128, 1>(bf16, 8))
                          : (bn == 64   ? variant<kGrad, 64, 2>(bf16, 9)
                             : bn == 96 ? variant<kGrad, 96, 2>(bf16, 10)
                                        : variant<kGrad, 128, 2>(bf16, 11));
        // one block holding every row copies only the rows that exist (rounded up to a
        // swizzle atom): the MMA's other rows are never stored
        const int box_a = ctas == 1 ? int(round_up(c.N, 8)) : BM, box_b = ctas == 1 ? 2 * bn : bn;
        CUtensorMap ta, tl, tb;
        const char *w = static_cast<const char *>(c.w) + first * c.w_stride * 2;
        if (!map16(&ta, c.x, c.N, c.H, c.x_stride * 2, BK, box_a, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !map16(&tb, w, cols, c.H, c.w_stride * 2, BK, box_b, CU_TENSOR_MAP_SWIZZLE_128B))
            return glu::cuda_fail(cudaErrorInvalidValue);
        tl = ta;
        if (plan.lists && !map16(&tl, at<char>(plan.listed), c.N, c.H, plan.listed_stride, BK, box_a,
                                 CU_TENSOR_MAP_SWIZZLE_128B))
            return glu::cuda_fail(cudaErrorInvalidValue);
        Params p{};
        p.cols = int(cols);
        p.depth = int(c.H);
        p.a_bytes = uint32_t(box_a) * BK * 2;
        p.target = c.distill ? nullptr : c.target;
        p.first = first;
        p.c1 = c1();
        if (grad) {
            p.out = at<char>(plan.g);
            p.out_stride = plan.g_stride;
            p.parts = plan.parts;
            p.part_cols = int(plan.part_cols);
            p.lse = c.lse;
            p.loss = c.loss;
            p.dloss = c.dloss;
            p.inv_t = inv_t();
            p.scale = scale();
        } else {
            p.part = at<float2>(plan.part);
            p.named = at<float>(plan.named);
            p.index = c.distill ? at<int>(plan.sorted) : nullptr;
            p.top = int(c.top);
        }
        return product(v, ta, tb, tl, ta, ta, p, c.N, c.H * 2, info);
    }

    int named(int64_t first, int64_t cols) const
    {
        NamedParams n{};
        n.count = count();
        n.rows = rows();
        n.sorted = at<int>(plan.sorted);
        n.order = at<int>(plan.order);
        n.entries = at<int>(plan.entries);
        n.share = at<float>(plan.share);
        n.top_logits = c.top_logits;
        n.lse = c.lse;
        n.dloss = c.dloss;
        n.scale = scale();
        n.N = int(c.N);
        n.top = int(c.top);
        n.first = first;
        n.cols = cols;
        n.c1 = c1();
        n.inv_t = inv_t();
        n.g = at<char>(plan.g);
        n.g_stride = plan.g_stride;
        n.parts = plan.parts;
        n.part_cols = plan.part_cols;
        void *args[] = {&n};
        const void *fn = bf16 ? reinterpret_cast<const void *>(&named_grad_kernel<__nv_bfloat16>)
                              : reinterpret_cast<const void *>(&named_grad_kernel<__half>);
        return launch(fn, unsigned(c.N), 128, 0, 1, args, s);
    }

    // Where a gradient product's result goes: a 16-bit matrix, or fp32 sums over the pieces; and the
    // parts of the tiles that are cut.
    int output(Params &p, CUtensorMap *to, CUtensorMap *tail, const CUtensorMap &unused, void *out, int64_t out_stride,
               int64_t r, int bn, int sums, int which) const
    {
        const auto f32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
        *to = *tail = unused;
        if (plan.tail_rows[which] > 0 && !make_map(tail, f32, at<char>(plan.tail[which]), plan.tail_rows[which], 2 * bn,
                                                   8 * bn, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B))
            return glu::cuda_fail(cudaErrorInvalidValue);
        p.sums = sums;
        if (sums) {
            if (!make_map(to, f32, at<char>(plan.sums), r, plan.ld, plan.ld * 4, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B))
                return glu::cuda_fail(cudaErrorInvalidValue);
            return GLU_OK;
        }
        p.out = static_cast<char *>(out);
        p.out_stride = out_stride * 2;
        p.vec_store = uintptr_t(out) % 32 == 0 && out_stride % 16 == 0  ? 32
                      : uintptr_t(out) % 16 == 0 && out_stride % 8 == 0 ? 16
                                                                        : 0;
        p.tma_store = p.vec_store && c.H % 8 == 0 &&
                      map16(to, out, r, c.H, out_stride * 2, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B);
        return GLU_OK;
    }

    // x transposed, of the rows that take part.
    int transpose() const
    {
        TransposeParams t{};
        t.x = static_cast<const char *>(c.x);
        t.listed = at<char>(plan.listed);
        t.x_stride = c.x_stride * 2;
        t.listed_stride = plan.listed_stride;
        t.count = count();
        t.N = int(c.N);
        t.H = int(c.H);
        t.out = at<char>(plan.xt);
        t.out_stride = plan.xt_stride;
        void *args[] = {&t};
        const int64_t h_tiles = (c.H + kTransTile - 1) / kTransTile;
        const dim3 grid(unsigned((c.N + kTransTile - 1) / kTransTile), unsigned(h_tiles < 65535 ? h_tiles : 65535));
        return launch(reinterpret_cast<const void *>(&transpose_kernel), grid, 256, 0, 1, args, s);
    }

    // dx (+)= g w over the piece.
    int data(int64_t first, int64_t cols, bool add, glu_launch_info_t *info) const
    {
        const int ctas = plan.ctas, bn = grad_bn(c.H);
        const Variant v = ctas == 1 ? (bn == 64 ? variant<kData, 64, 1>(bf16, 12) : variant<kData, 128, 1>(bf16, 13))
                                    : (bn == 64 ? variant<kData, 64, 2>(bf16, 14) : variant<kData, 128, 2>(bf16, 15));
        const int box_a = ctas == 1 ? int(round_up(c.N, 8)) : BM;
        CUtensorMap ta, t2, tb, to, tt;
        const char *w = static_cast<const char *>(c.w) + first * c.w_stride * 2;
        const uint64_t second = plan.parts == 2 ? uint64_t(plan.part_cols) * 2 : 0;
        if (!map16(&ta, at<char>(plan.g), c.N, cols, plan.g_stride, BK, box_a, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !map16(&t2, at<char>(plan.g + second), c.N, cols, plan.g_stride, BK, box_a, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !map16(&tb, w, cols, c.H, c.w_stride * 2, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B))
            return glu::cuda_fail(cudaErrorInvalidValue);
        Params p{};
        p.cols = int(c.H);
        // every piece is cut alike, so that their sums meet: a last, shorter one reads zeros past its end
        p.depth = int(plan.piece);
        p.a_bytes = uint32_t(box_a) * BK * 2 * uint32_t(plan.parts);
        p.scale = scale();
        p.parts = plan.parts;
        p.cut = cuts();
        if (int st = output(p, &to, &tt, ta, c.dx, c.dx_stride, c.N, bn, plan.pieces == 1 ? 0 : add ? 2 : 1, 0))
            return st;
        if (int st = product(v, ta, tb, t2, to, tt, p, c.N, plan.g_stride, info)) return st;
        if (first + cols < c.V) return GLU_OK;
        return sum(p, v, false, c.dx, c.dx_stride);
    }

    // dw = g^T x for the piece.
    int weight(int64_t first, int64_t cols, glu_launch_info_t *info) const
    {
        const int bn = grad_bn(c.H);
        const Variant v = plan.transpose
                              ? (bn == 64 ? variant<kWeightT, 64, 2>(bf16, 20) : variant<kWeightT, 128, 2>(bf16, 21))
                              : (bn == 64 ? variant<kWeight, 64, 2>(bf16, 16) : variant<kWeight, 128, 2>(bf16, 17));
        CUtensorMap ta, tb, tl, to, tt;
        // columns behind the piece's are rows of dw that do not exist
        if (!map16(&ta, at<char>(plan.g), c.N, (plan.parts - 1) * plan.part_cols + cols, plan.g_stride, 64, BK,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
            !(plan.transpose
                  ? map16(&tb, at<char>(plan.xt), c.H, round_up(c.N, 64), plan.xt_stride, BK, bn,
                          CU_TENSOR_MAP_SWIZZLE_128B)
                  : map16(&tb, c.x, c.N, c.H, c.x_stride * 2, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B)) ||
            !map16(&tl, at<char>(plan.listed), c.N, c.H, plan.listed_stride, 64, BK, CU_TENSOR_MAP_SWIZZLE_128B))
            return glu::cuda_fail(cudaErrorInvalidValue);
        Params p{};
        p.cols = int(c.H);
        p.m_rows = int(cols);
        p.a_bytes = uint32_t(BM * BK * 2);
        p.scale = scale();
        p.parts = plan.parts;
        p.part_cols = int(plan.part_cols);
        p.cut = cuts() + (first + cols < c.V ? 1 : 2);
        char *out = static_cast<char *>(c.dw) + first * c.dw_stride * 2;
        if (int st = output(p, &to, &tt, ta, out, c.dw_stride, cols, bn, 0, 1)) return st;
        if (int st = product(v, ta, tb, tl, to, tt, p, cols, c.N * 2, info)) return st;
        return sum(p, v, true, out, c.dw_stride);
    }

    // What the product `p` left as sums, where it can have left any.
    int sum(const Params &p, const Variant &v, bool weight, void *out, int64_t out_stride) const
    {
        const int tile_m = BM * v.ctas;
        const int64_t m_blocks = ((weight ? int64_t(p.m_rows) : c.N) + tile_m - 1) / tile_m;
        const int64_t tiles = m_blocks * p.n_blocks;
        // A cut saves less than a round: none from 26 rounds on.  How many rows take
        // part, which counts the tiles of dx and the slices of dw, only the GPU knows.
        const int64_t k_tiles = weight ? p.parts * ((c.N + BK - 1) / BK) : (p.depth + BK - 1) / BK;
        const int slots = kSms / v.ctas;
        const bool cut = k_tiles >= 8 && (!weight || (tiles % slots != 0 && tiles < 26 * slots));
        if (!p.sums && !cut) return GLU_OK;
        SumParams q{};
        q.tail = at<float>(plan.tail[weight]);
        q.sums = p.sums ? at<float>(plan.sums) : nullptr;
        q.ld = plan.ld;
        q.count = count();
        q.rows = rows();
        q.weight = weight;
        q.N = int(c.N);
        q.cols = p.cols;
        q.m_rows = p.m_rows;
        q.n_blocks = p.n_blocks;
        q.group_m = p.group_m;
        q.cut = p.cut;
        q.tile_m = tile_m;
        q.tile_n = 2 * v.bn;
        q.scale = scale();
        q.out = static_cast<char *>(out);
        q.out_stride = out_stride * 2;
        void *args[] = {&q};
        const int64_t most = p.sums ? tiles : (tiles < 2 * slots ? tiles : 2 * slots);
        const int64_t blocks = most * tile_m * v.bn / 2 / 256;
        const void *fn = bf16 ? reinterpret_cast<const void *>(&sum_kernel<__nv_bfloat16>)
                              : reinterpret_cast<const void *>(&sum_kernel<__half>);
        return launch(fn, unsigned(blocks < 16 * sms ? blocks : 16 * sms), 256, 0, 1, args, s);
    }

    int forward(glu_launch_info_t *info) const
    {
        if (c.distill)
            if (int st = teacher()) return st;
        if (plan.lists)
            if (int st = list()) return st;
        if (int st = logits(false, 0, c.V, info)) return st;
        JoinParams j{};
        j.part = at<float2>(plan.part);
        j.n_parts = 2 * int((c.V + 2 * plan.bn - 1) / (2 * plan.bn));
        j.N = int(c.N);
        j.count = plan.lists ? count() : nullptr;
        j.rows = rows();
        j.target = c.distill ? nullptr : c.target;
        j.V = c.V;
        j.named = at<float>(plan.named);
        j.c1 = c1();
        j.loss = c.loss;
        j.lse = c.lse;
        if (c.distill) {
            j.share = at<float>(plan.share);
            j.order = at<int>(plan.order);
            j.entries = at<int>(plan.entries);
            j.neg_entropy = at<float>(plan.entropy);
            j.top = int(c.top);
            j.top_logits = c.top_logits;
        }
        void *args[] = {&j};
        // 32 rows a block read whole lines; 8 rows while that is what it takes to fill the GPU
        // (forward of 64 x 4096, 32768 tokens: 51.2 -> 49.1 us, with w's prefetch)
        const bool wide = c.N > 8 * kSms * 2;
        return launch(wide ? reinterpret_cast<const void *>(&join_kernel<32>)
                           : reinterpret_cast<const void *>(&join_kernel<8>),
                      unsigned((c.N + (wide ? 31 : 7)) / (wide ? 32 : 8)), kJoinThreads, 0, 1, args, s);
    }

    int backward(glu_launch_info_t *info) const
    {
        if (c.distill)
            if (int st = teacher()) return st;
        if (int st = list()) return st;
        if (plan.transpose)
            if (int st = transpose()) return st;
        for (int i = 0; i < plan.pieces; ++i) {
            const int64_t first = i * plan.piece, cols = c.V - first < plan.piece ? c.V - first : plan.piece;
            if (int st = logits(true, first, cols, info)) return st;
            if (c.distill)
                if (int st = named(first, cols)) return st;
            // dx first: it finds what g's product read last of w in L2
            if (c.dx)
                if (int st = data(first, cols, i > 0, info)) return st;
            if (c.dw)
                if (int st = weight(first, cols, info)) return st;
        }
        return GLU_OK;
    }
};

int run(Call c, glu_stream_t stream)
{
    bool empty = false;
    if (int st = validate(c, &empty)) return st;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (empty) {
        if (c.backward && c.dw) {       // no rows: dw = 0
            const cudaError_t e =
                cudaMemset2DAsync(c.dw, size_t(c.dw_stride) * 2, 0, size_t(c.H) * 2, size_t(c.V), s);
            if (e != cudaSuccess) {
                (void)cudaGetLastError();
                return glu::cuda_fail(e);
            }
        }
        glu::record_launch(glu_launch_info_t{});
        return GLU_OK;
    }
    Plan plan;
    if (!plan_for(c, c.workspace_bytes, &plan)) return GLU_ERR_WORKSPACE;
    Run r{c, plan};
    if (int st = device(&r.dev, &r.sms)) return st;
    if (int st = check_device(c, r.dev)) return st;
    r.s = s;
    r.bf16 = c.dtype == GLU_BF16;
    r.ws = static_cast<char *>(c.workspace);
    r.type16 = r.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    glu_launch_info_t info{};
    if (int st = c.backward ? r.backward(&info) : r.forward(&info)) return st;
    info.backward = c.backward;
    info.path = c.distill ? 14 : 13;
    glu::record_launch(info);
    return GLU_OK;
}

size_t workspace_bytes(int64_t N, int64_t H, int64_t V, int64_t top, bool backward)
{
    Call c{};
    if (N < 1 || H < 1 || V < 1 || N > kMaxSize || H > kMaxSize || V > kMaxSize || top < 0 || top > kMaxTop) return 0;
    c.N = N;
    c.H = H;
    c.V = V;
    c.top = top;
    c.distill = top > 0;
    c.backward = backward;
    if (backward) {             // room for both gradients
        c.dx = &c;
        c.dw = &c;
    }
    Plan p;
    (void)plan_for(c, UINT64_MAX, &p);
    return size_t(p.bytes);
}

}  // namespace
}  // namespace loss
}  // namespace glu

extern "C" int glu_linear_ce_fwd(const void *x, int64_t x_stride, const void *w, int64_t w_stride,
                                 const int64_t *target, float *loss, float *lse, int64_t N, int64_t H, int64_t V,
                                 glu_dtype_t dtype, void *workspace, size_t workspace_bytes, glu_stream_t stream)
{
    glu::loss::Call c{};
    c.x = x;
    c.x_stride = x_stride;
    c.w = w;
    c.w_stride = w_stride;
    c.N = N;
    c.H = H;
    c.V = V;
    c.dtype = dtype;
    c.target = target;
    c.temperature = 1.0f;
    c.loss = loss;
    c.lse = lse;
    c.workspace = workspace;
    c.workspace_bytes = workspace_bytes;
    return glu::loss::run(c, stream);
}

extern "C" int glu_linear_ce_bwd(const float *dloss, const void *x, int64_t x_stride, const void *w, int64_t w_stride,
                                 const int64_t *target, const float *loss, const float *lse, void *dx,
                                 int64_t dx_stride, void *dw, int64_t dw_stride, int64_t N, int64_t H, int64_t V,
                                 glu_dtype_t dtype, void *workspace, size_t workspace_bytes, glu_stream_t stream)
{
    glu::loss::Call c{};
    c.x = x;
    c.x_stride = x_stride;
    c.w = w;
    c.w_stride = w_stride;
    c.N = N;
    c.H = H;
    c.V = V;
    c.dtype = dtype;
    c.target = target;
    c.temperature = 1.0f;
    c.loss = const_cast<float *>(loss);
    c.lse = const_cast<float *>(lse);
    c.dloss = dloss;
    c.dx = dx;
    c.dx_stride = dx_stride;
    c.dw = dw;
    c.dw_stride = dw_stride;
    c.workspace = workspace;
    c.workspace_bytes = workspace_bytes;
    c.backward = true;
    return glu::loss::run(c, stream);
}

extern "C" int glu_linear_distill_fwd(const void *x, int64_t x_stride, const void *w, int64_t w_stride,
                                      const int64_t *index, int64_t index_stride, const void *logit,
                                      int64_t logit_stride, float temperature, float *loss, float *lse,
                                      float *top_logits, int64_t N, int64_t H, int64_t V, int64_t K,
                                      glu_dtype_t dtype, glu_dtype_t logit_dtype, void *workspace,
                                      size_t workspace_bytes, glu_stream_t stream)
{
    glu::loss::Call c{};
    c.x = x;
    c.x_stride = x_stride;
    c.w = w;
    c.w_stride = w_stride;
    c.N = N;
    c.H = H;
    c.V = V;
    c.dtype = dtype;
    c.distill = true;
    c.index = index;
    c.index_stride = index_stride;
    c.logit = logit;
    c.logit_stride = logit_stride;
    c.logit_dtype = logit_dtype;
    c.top = K;
    c.temperature = temperature;
    c.loss = loss;
    c.lse = lse;
    c.top_logits = top_logits;
    c.workspace = workspace;
    c.workspace_bytes = workspace_bytes;
    return glu::loss::run(c, stream);
}

extern "C" int glu_linear_distill_bwd(const float *dloss, const void *x, int64_t x_stride, const void *w,
                                      int64_t w_stride, const int64_t *index, int64_t index_stride,
                                      const void *logit, int64_t logit_stride, float temperature, const float *lse,
                                      const float *top_logits, void *dx, int64_t dx_stride, void *dw,
                                      int64_t dw_stride, int64_t N, int64_t H, int64_t V, int64_t K,
                                      glu_dtype_t dtype, glu_dtype_t logit_dtype, void *workspace,
                                      size_t workspace_bytes, glu_stream_t stream)
{
    glu::loss::Call c{};
    c.x = x;
    c.x_stride = x_stride;
    c.w = w;
    c.w_stride = w_stride;
    c.N = N;
    c.H = H;
    c.V = V;
    c.dtype = dtype;
    c.distill = true;
    c.index = index;
    c.index_stride = index_stride;
    c.logit = logit;
    c.logit_stride = logit_stride;
    c.logit_dtype = logit_dtype;
    c.top = K;
    c.temperature = temperature;
    c.lse = const_cast<float *>(lse);
    c.top_logits = const_cast<float *>(top_logits);
    c.dloss = dloss;
    c.dx = dx;
    c.dx_stride = dx_stride;
    c.dw = dw;
    c.dw_stride = dw_stride;
    c.workspace = workspace;
    c.workspace_bytes = workspace_bytes;
    c.backward = true;
    return glu::loss::run(c, stream);
}

extern "C" size_t glu_linear_ce_workspace_bytes(int64_t N, int64_t H, int64_t V, int backward)
{
    return glu::loss::workspace_bytes(N, H, V, 0, backward != 0);
}

extern "C" size_t glu_linear_distill_workspace_bytes(int64_t N, int64_t H, int64_t V, int64_t K, int backward)
{
    return K < 1 ? 0 : glu::loss::workspace_bytes(N, H, V, K, backward != 0);
}
