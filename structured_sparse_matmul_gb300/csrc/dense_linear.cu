// Dense products of 16-bit operands on the tensor cores, with what follows them
// in the epilogue:
//
//   Y[t][r] = act(sum_k X[t][k] W[r][k] + bias[r]) + residual[t][r]
//   Y[t][r] = act(G) * U,  G = X . Wg^T, U = X . Wu^T     (the gated pair)
//
// Either operand may be stored with K along its rows or along its columns: the
// tensor memory copies bring 64 x 64 boxes of the latter, and the MMAs read both
// orders from shared memory, so that the gradients dY . W and dY^T . X need no
// transposed copy. Two products that add up to one output (dG . Wg + dU . Wu) are one
// product over both K; two that share an operand (dG^T . X, dU^T . X) are one grid.
//
// dense_pair_kernel, many tokens: pairs of CTAs (cta_group::2), 256 rows of X by up to 256 of W
// a tile (each CTA loads its own 128 rows of X and half of W's; of a gated pair, the
// first CTA loads Wg's and the second Wu's rows, and a tile is 128 features of
// both), persistent, two TMEM accumulators of 256 columns, so that a tile's
// epilogue runs under the next one's MMAs.
//   warp 0     TMA producer: six stages of 64 elements of K, 128B swizzle.
//   warp 1     TMEM owner, MMA issuer (one thread of the first CTA).
//   warps 4..  epilogue: 32 rows x half of the columns a warp. A lane has a row, 16 columns at a time; bias,
//              activation, rounding; then into boxes of 32 rows x 64 bytes, which tensor memory stores bring out
//              (a residual's boxes came in by the same way). Of a CTA's last tile, which nothing hides, fp32 sums that
//              need no more than a residual go to the boxes straight from the registers, all of them at once (4096 x 1024
//              over 8192 53.5 us through the loop and 48.5 so).
// The residual is added to the whole sum. (Sums of several chunks that start from it, read under the MMAs, are rounded to
// its spacing once a chunk: 2^24 and eight ones were 2^24. Read late it costs a wait where nothing hides it and less
// elsewhere, us: 2048 x 2048 over 2048 18.4 then and 20.6 now, 4096 x 1024 over 8192 48.7 and 49.2, 4096 x 4096 over 8192
// 205 and 188, 8192 x 8192 over 2048 313 and 224.)
// Where the outputs' rows do not start and end on 16 bytes, the boxes are copied out by the warps. With
// few tiles, K is split over the pairs of a cluster, which copy their sums to each other at the end.
//
// Measured, bf16 (us; in brackets the operations at the measured rate of a library product):
// 8192 x 4096 over 11008 with residual 387 (383), 8192 x 11008 over 4096 gated with 8-bit checkpoints 776 (766), 450 and 899 at
// the 1500 MHz that the power cap leaves after some hundred ms; dX of that,
// 8192 x 4096 over 2 x 11008, 784 (766), dWg and dWu 822 (766). Bound by the MMAs: a K block takes 0.285 us, theirs is 0.27.
// Products of fewer tiles than pairs wait for L2 as well: 64 KB a pair and K block, 10.3 TB/s of all.
//
// dense_narrow_kernel, few tokens or few tiles: W on the MMA's M side (its rows fill the
// tensor cores' rows), 16 to 128 tokens a tile, two CTAs an SM, K over the CTAs of a cluster,
// which add their sums up through distributed shared memory in rank order. 517 x 1001 over 1041 takes 10.8 us: W is
// read again for every 32 tokens, 36 MB from L2 at 10 TB/s, and a launch, the ring's first loads and
// the stores of rows of odd length. (A ring twice as deep, one CTA an SM, was 2 to 19 % slower in 30 of 44 products: the
// next launch's setup no longer runs beside this one's end.)
//
// The tensor cores' fp32 sums truncate: over K they lose about K * 2^-30 of
// random sums and six times that of sums of one sign (measured: 9e-6 and 5e-5 at
// K = 8192). To fp32 outputs, and to the largest magnitude of a group of 8-bit checkpoints, that is much:
// there the sums are taken out every kChunk elements of K and added in registers. Next to a rounding to 16 bits
// it is little up to kLongChunk.
#include <algorithm>
#include <atomic>

#include "vnm_dense16.cuh"
#include "vnm_internal.h"
#include "vnm_ptx.cuh"

namespace vnm {
namespace {

constexpr int kTile = 128;        // rows of an operand in a CTA's stage
constexpr int kBlockK = 64;       // elements of K in a stage: 128 bytes
constexpr int kOperandBytes = kTile * 128;
constexpr int kChunk = 1024 / kBlockK, kLongChunk = 32768 / kBlockK;
constexpr int kMaxSplits = 8, kMaxPairSplits = 4;
constexpr int kMaxDevicesDl = 64;
constexpr int kGroupM = 8;

struct Maps {
    CUtensorMap x[2], w[2];
};

// Of pairs' outputs and residuals, where their rows start on 16 bytes.
struct OutMaps {
    CUtensorMap y[2], g, u, res[2];
};

struct GemmArgs {
    OutArgs o;
    int kind;
    int num_kb;       // K blocks of one product
    int total_kb;     // of an output's sum
    int chunk_kb;     // K blocks of one TMEM sum
    int x_tiles;      // tiles of X's rows, of one product
    int m_tiles, n_tiles, tiles;
    int stages, stage_bytes;  // of pairs
    int tile_n;       // of pairs: rows of W of a tile (of a gated pair, half of them Wg's and half Wu's)
    int splits, kb_per_split;
    bool x_t, w_t;
    uint32_t idesc;
    bool beside, next_beside;
    int* status;
    int skip_stage;
};

// Instruction descriptor of kind::f16 with an fp32 accumulator: bits 4-5 D format (1 = f32),
// 7-9 / 10-12 A / B format (0 = f16, 1 = bf16), 15 / 16 A / B major-ness (1 = M/N-major),
// 17-22 N >> 3, 24-28 M >> 4.
constexpr uint32_t f16_idesc(int m, int n, bool bf16, bool a_mn, bool b_mn) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// D[tmem] (+)= A[smem] x B[smem]; of a pair, each CTA holding half the rows of A, of B and of D.
__device__ __forceinline__ void tc_mma_f16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on `bar` of both CTAs of the pair whose first CTA has rank `lead` in the cluster, when the
// MMAs issued so far are done.
__device__ __forceinline__ void tc_commit_pair(uint32_t bar, int lead) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3 << lead))
        : "memory");
}

// Brings `bytes` (a multiple of 16) from `p` (16-byte aligned) into L2.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// `bytes` of this CTA's shared memory to that of a CTA of the cluster, counted on a barrier there.
__device__ __forceinline__ void copy_to_cluster(uint32_t cluster_dst, uint32_t src, uint32_t bytes, uint32_t cluster_bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(cluster_dst),
                 "r"(src), "r"(bytes), "r"(cluster_bar)
                 : "memory");
}

// An operand's 128 x 64 part of a stage in shared memory, 128B swizzle. K along the rows: 128-byte
// rows, 8-row groups 1024 bytes apart; an MMA (16 of K) takes 32 bytes of every row.
// Transposed: two boxes of 64 operand rows, 8192 bytes apart; in a box 128-byte lines of
// one k, 8-line groups 1024 bytes apart; an MMA takes 16 lines.
__device__ __forceinline__ uint64_t operand_desc(uint32_t at, bool transposed) {
    return make_smem_desc(at, transposed ? 8192 : 16, 1024, kLayoutSw128);
}
__device__ __forceinline__ uint32_t operand_step(bool transposed) { return transposed ? 2048 / 16 : 32 / 16; }

// The tile's place: tiles of X's rows in groups of kGroupM, those fastest, so that the CTAs
// that run together share a few tiles of both operands in L2.
__device__ __forceinline__ void tile_at(const GemmArgs& a, int tile, int& mt, int& nt) {
    const int per_group = kGroupM * a.n_tiles;
    const int g = tile / per_group, r = tile - g * per_group;
    const int rows = min(kGroupM, a.m_tiles - g * kGroupM);
    nt = r / rows;
    mt = g * kGroupM + (r - nt * rows);
}

// Status words of the calls that were given none (of the device's all).
__device__ int g_status[3];

__device__ __forceinline__ float4 ld_shared_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_v2(uint32_t addr, float x, float y) {
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ void st_shared_f4(uint32_t addr, float a, float b, float c, float d) {
    st_shared_v4(addr, __float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
}

// ------------------------------------------------------------------ pairs of CTAs

// 6 stages of 128 rows of X and 128 of W, or more of less: a stage's way round (loads of a microsecond, its MMAs, the
// barriers) takes 1.4 us, its MMAs 0.27 (a K block took 0.42, 0.35 and 0.285 us with 3, 4 and 5 stages).
constexpr int kPairRing = 192 * 1024;
constexpr int kPairMaxStages = 8;
constexpr int kPairHelpers = 4, kPairEpilogue = 8;
constexpr int kPairThreads = 32 * (kPairHelpers + kPairEpilogue);
// A warp's staged outputs: two boxes of 32 rows x 64 bytes. Of a gated pair a box holds 32 rows x 32 features
// of Y, and with 8-bit checkpoints theirs (one box), or 16 features of Y and of 16-bit checkpoints (one).
constexpr int kStageOut = 4096;
constexpr int kSumBytes = kTile * 1024;  // a split's sums of a CTA's rows; the rest of the memory takes the other pairs'
constexpr int kPairSmem = kPairRing + kPairEpilogue * kStageOut + 1024;
static_assert(kSumBytes + (kMaxPairSplits - 1) * (kTile / kMaxPairSplits) * 1024 <= kPairRing + kPairEpilogue * kStageOut &&
                  kSumBytes + 2 * ((kTile + 2) / 3) * 1024 <= kPairRing + kPairEpilogue * kStageOut,
              "the splits' sums fit");
static_assert(kPairRing / kPairEpilogue >= 16 * 1024, "a warp's last boxes: 32 rows x 128 columns of fp32");
static_assert(kPairSmem > 116 * 1024 && kPairSmem <= 226 * 1024, "one CTA an SM: each holds all of its TMEM");
// Registers of the variant that adds chunks up: 128 sums and a load of 32 columns do not fit the 168 that
// 12 warps get; the epilogue takes what the helper warps leave (in warps: 4 x 56 + 8 x 224 = 12 x 168).
// Where K is split, the code after the sums runs on all warps, and the loads are of 16 columns instead.
constexpr int kSumLaunchRegs = 168, kSumHelperRegs = 56, kSumAddRegs = 224;
static_assert(kPairHelpers * kSumHelperRegs + kPairEpilogue * kSumAddRegs == (kPairHelpers + kPairEpilogue) * kSumLaunchRegs,
              "register shares");

// 16-byte piece j of row `row` of a box of RB-byte rows in shared memory, in the order of the tensor memory copies'
// swizzle for that width (a warp's lanes, a row each, then write to all banks alike).
template <int RB>
__device__ __forceinline__ uint32_t box_piece(uint32_t buf, int row, int j) {
    const int flip = RB == 128 ? row & 7 : RB == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
    return buf + RB * row + 16 * (j ^ flip);
}

// Piece j and column c of row `row` of a split's fp32 sums, 256 columns a row.
__device__ __forceinline__ uint32_t sum_piece(uint32_t base, int row, int j) { return base + 1024 * row + 16 * (j ^ (row & 7)); }
__device__ __forceinline__ uint32_t sum_at(uint32_t base, int row, int c) { return sum_piece(base, row, c >> 2) + 4 * (c & 3); }

// A staged box (the first `rows` rows, `bytes` bytes of each) to memory of any alignment of its elements (G bytes; row 0
// at `to`), by a warp, a 4-byte word a lane: whole where the rows all start on 4 bytes, else element by element (putting
// a word of memory together from two staged ones took twice as long). Apart from the epilogue's loop: its
// code there, fetched for every tile, made the tiles that do not need it 40 % slower.
template <int RB, int G>
__device__ __noinline__ void copy_box(uint8_t* to, int64_t pitch, int rows, int bytes, uint32_t buf, int lane) {
    constexpr int kPer = RB / 4, kRows = 32 / kPer;  // lanes of a row, rows at a time
    const int w = lane % kPer, r = lane / kPer;
    const bool words = ((reinterpret_cast<uintptr_t>(to) | static_cast<uintptr_t>(pitch)) & 3) == 0;
    to += r * pitch + 4 * w;
    const int left = bytes - 4 * w;
#pragma unroll 4
    for (int row0 = 0; row0 < 32; row0 += kRows) {
        uint32_t x;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(box_piece<RB>(buf, row0 + r, w >> 2) + 4 * (w & 3)) : "memory");
        const bool here = row0 + r < rows;
        if (G == 4 || (words && left >= 4)) {
            if (here && left >= 4) *reinterpret_cast<uint32_t*>(to) = x;
        } else {
#pragma unroll
            for (int e = 0; e < 4; e += G) {
                if (!here || e >= left) continue;
                if (G == 2)
                    *reinterpret_cast<uint16_t*>(to + e) = static_cast<uint16_t>(x >> (8 * e));
                else
                    to[e] = static_cast<uint8_t>(x >> (8 * e));
            }
        }
        to += kRows * pitch;
    }
}

// A staged box of elements of G bytes to rows m0 .., columns n0 .. n0 + RB / G - 1 (below `end`) of a matrix. All lanes have
// written their rows.
template <int RB, int G, bool ALIGNED>
__device__ __forceinline__ void emit_box(const CUtensorMap* tm, bool tma, void* p, int64_t ld, int64_t m0, int64_t n0, int64_t T,
                                         int64_t end, uint32_t buf, int lane) {
    if (m0 >= T || n0 >= end) return;
    // (a tensor memory store that ends inside 16 bytes writes all of them)
    if (ALIGNED || (tma && (n0 + RB / G <= end || end * G % 16 == 0))) {
        if (lane == 0) tma_store_2d(tm, static_cast<int32_t>(n0), static_cast<int32_t>(m0), buf);
    } else {
        copy_box<RB, G>(static_cast<uint8_t*>(p) + (m0 * ld + n0) * G, ld * G, static_cast<int>(min(static_cast<int64_t>(32), T - m0)),
                        static_cast<int>(min(static_cast<int64_t>(RB), (end - n0) * G)), buf, lane);
    }
}

__device__ __forceinline__ bool all_vec(const OutArgs& o) { return o.y_vec && o.res_vec && o.keep_vec; }

// A row's 16 columns of the residual as they are stored.
struct Raw16 {
    Raw8 h[2];
};

// SUM: the sums are taken out every chunk_kb K blocks and added up in registers; SPLIT: K is split over
// the pairs of a cluster, one tile a cluster; ALIGNED: the outputs' and the residual's rows start on 16 bytes (the
// code for others, in the same loop, costs the aligned ones a third of their epilogue) and end on 16.
template <bool GATED, bool SUM, bool SPLIT, bool ALIGNED>
__global__ void __launch_bounds__(kPairThreads, 1)
    dense_pair_kernel(const __grid_constant__ Maps maps, const __grid_constant__ OutMaps outs, const __grid_constant__ GemmArgs a) {
    static_assert(SUM || !SPLIT, "a split's sums are held in registers until the ring is free");
    constexpr int LD = SPLIT ? 16 : 32;
    constexpr bool kSplitRegs = SUM && !SPLIT;
    constexpr int kTileN = GATED ? 128 : 256;  // columns of Y of a tile
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[kPairMaxStages];   // the stage has landed in both CTAs (the first CTA's)
    __shared__ __align__(8) uint64_t empty_bar[kPairMaxStages];  // its MMAs are done
    __shared__ __align__(8) uint64_t accf_bar[2];    // the TMEM sum is complete
    __shared__ __align__(8) uint64_t acce_bar[2];    // and has been read by both CTAs (the first CTA's)
    // of each epilogue warp's two output boxes: the residual's box has landed in it
    __shared__ __align__(8) uint64_t res_bar[GATED ? 1 : kPairEpilogue][2];
    __shared__ __align__(8) uint64_t split_bar;  // the other pairs' sums of this CTA's rows have landed
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int ST = a.stages, stage_bytes = a.stage_bytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x & 1);  // of the pair
    const int cluster = SPLIT ? 2 * a.splits : 2;       // CTAs of the cluster
    const int pair = SPLIT ? (static_cast<int>(blockIdx.x) % cluster) >> 1 : 0, lead_rank = 2 * pair;
    const int tile0 = static_cast<int>(blockIdx.x) / cluster;
    const int tile_step = SPLIT ? a.tiles : static_cast<int>(gridDim.x >> 1);
    const int kb_first = SPLIT ? min(a.total_kb, pair * a.kb_per_split) : 0;
    const int kb_last = SPLIT ? min(a.total_kb, kb_first + a.kb_per_split) : a.total_kb;

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(smem_u32(&full_bar[s]), 1);
            mbar_init(smem_u32(&empty_bar[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&accf_bar[s]), 1);
            mbar_init(smem_u32(&acce_bar[s]), 2 * kPairEpilogue);
            for (int w = 0; !GATED && w < kPairEpilogue; ++w) mbar_init(smem_u32(&res_bar[w][s]), 1);
        }
        mbar_init(smem_u32(&split_bar), 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc_group<2>(smem_u32(&tmem_slot), 512);
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();  // the CTAs' barriers and TMEM exist
    tc_fence_after_sync();
    after_the_one_before(a.beside, a.o.res[0] != nullptr);
    let_next_grid_start();
    const uint32_t tmem = tmem_slot;
    volatile int* abort = &abort_flag;

    if (kSplitRegs && warp < kPairHelpers) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kSumHelperRegs));
    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        int it = 0, slot = 0;
        uint32_t phase = 1;
        bool run = true;
        for (int tile = tile0; tile < a.tiles && run; tile += tile_step) {
            int mt, nt;
            tile_at(a, tile, mt, nt);
            const int seg = a.kind == kTwoByRows && mt >= a.x_tiles ? 1 : 0;
            const int xrow = ((mt - seg * a.x_tiles) * 2 + rank) * kTile;
            const int wrows = a.tile_n / 2, wrow = GATED ? nt * wrows : nt * a.tile_n + rank * wrows;
            const uint32_t wbytes = a.w_t ? (wrows > 64 ? 16384 : 8192) : wrows * 128;
            for (int kb = kb_first; kb < kb_last; ++kb, ++it) {
                if (!mbar_wait_warp(smem_u32(&empty_bar[slot]), phase, abort)) {
                    run = false;
                    break;
                }
                if (elect_one() && (it != a.skip_stage || blockIdx.x != 0)) {
                    const bool second = kb >= a.num_kb;  // of a sum of two
                    const CUtensorMap* tx = &maps.x[second || seg];
                    const CUtensorMap* tw = &maps.w[GATED ? rank : second];
                    const int k = (second ? kb - a.num_kb : kb) * kBlockK;
                    const uint32_t sx = smem_base + slot * stage_bytes, sw = sx + kOperandBytes;
                    const uint32_t fb = smem_u32(&full_bar[slot]), lead = dsmem_map(fb, lead_rank);
                    // the second CTA's bytes may arrive before the first CTA expects them: the
                    // phase cannot end before that CTA's own arrival
                    if (rank == 0) mbar_arrive_expect_tx(fb, 2 * (kOperandBytes + wbytes));
                    if (a.x_t) {
                        tma_load_2d_pair(sx, tx, xrow, k, lead);
                        tma_load_2d_pair(sx + 8192, tx, xrow + 64, k, lead);
                    } else {
                        tma_load_2d_pair(sx, tx, k, xrow, lead);
                    }
                    if (a.w_t) {
                        tma_load_2d_pair(sw, tw, wrow, k, lead);
                        if (wrows > 64) tma_load_2d_pair(sw + 8192, tw, wrow + 64, k, lead);
                    } else {
                        tma_load_2d_pair(sw, tw, k, wrow, lead);
                    }
                }
                __syncwarp();
                if (++slot == ST) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
        if (*abort) {
            // every copy issued must land before the CTA exits; the second CTA of a pair has no
            // barrier of its own to wait on, and gives its copies a millisecond
            if (rank == 0) {
                for (int k = it > ST ? it - ST : 0; k < it; ++k)
                    if (k != a.skip_stage || blockIdx.x != 0)
                        mbar_drain(smem_u32(&full_bar[k % ST]), static_cast<uint32_t>(k / ST) & 1u);
            } else {
                const uint64_t t0 = global_timer_ns();
                for (int i = 0; i < (1 << 20) && global_timer_ns() - t0 < 1000000; ++i) __nanosleep(1000);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        const uint64_t xdesc = operand_desc(smem_base, a.x_t), wdesc = operand_desc(smem_base + kOperandBytes, a.w_t);
        const uint32_t xstep = operand_step(a.x_t), wstep = operand_step(a.w_t);
        int it = 0, slot = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 1;
        bool run = rank == 0;
        for (int tile = tile0; tile < a.tiles && run; tile += tile_step) {
            for (int kb0 = kb_first; kb0 < kb_last && run; kb0 += a.chunk_kb) {
                const int kb1 = min(kb_last, kb0 + a.chunk_kb);
                if (!mbar_wait_warp(smem_u32(&acce_bar[acc]), acc_phase, abort)) {
                    run = false;
                    break;
                }
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    if (!mbar_wait_warp(smem_u32(&full_bar[slot]), phase, abort)) {
                        run = false;
                        break;
                    }
                    tc_fence_after_sync();
                    if (elect_one()) {
                        const uint64_t off = static_cast<uint64_t>((slot * stage_bytes) >> 4);
#pragma unroll
                        for (uint32_t s = 0; s < 4; ++s)
                            tc_mma_f16_pair(tmem + acc * 256, xdesc + off + s * xstep, wdesc + off + s * wstep, a.idesc,
                                            kb > kb0 || s > 0 ? 1u : 0u);
                        tc_commit_pair(smem_u32(&empty_bar[slot]), lead_rank);
                        if (kb + 1 == kb1) tc_commit_pair(smem_u32(&accf_bar[acc]), lead_rank);
                    }
                    __syncwarp();
                    if (++slot == ST) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1;
                }
            }
        }
        // every MMA issued is done before TMEM goes back
        if (it > 0) mbar_drain(smem_u32(&empty_bar[(it - 1) % ST]), static_cast<uint32_t>((it - 1) / ST) & 1u);
    } else if (warp >= kPairHelpers) {
        // ------------------------------------------------ epilogue
        if (kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumAddRegs));
        const OutArgs& o = a.o;
        const int quarter = warp & 3, half = (warp - kPairHelpers) >> 2;  // TMEM lanes 32 quarter ..; columns
        const uint32_t lane_addr = static_cast<uint32_t>(32 * quarter) << 16;
        const uint32_t acce_lead = dsmem_map(smem_u32(&acce_bar[0]), lead_rank);
        const uint32_t stage = smem_base + kPairRing + (warp - kPairHelpers) * kStageOut;
        int acc = 0, box = 0;
        uint32_t acc_phase = 0, res_phase = 0, res_pending = 0;
        bool run = true;
        auto wait_sum = [&] {
            run = mbar_wait_warp(smem_u32(&accf_bar[acc]), acc_phase, abort);
            tc_fence_after_sync();
            return run;
        };
        auto release = [&] {  // all read: the MMAs may have the sum's columns back
            tc_fence_before_sync();
            __syncwarp();
            if (elect_one()) mbar_arrive_cluster(acce_lead + 8 * acc);
            if (++acc == 2) {
                acc = 0;
                acc_phase ^= 1;
            }
        };
        for (int tile = tile0; tile < a.tiles && run; tile += tile_step) {
            int mt, nt;
            tile_at(a, tile, mt, nt);
            const int seg = a.kind == kTwoByRows && mt >= a.x_tiles ? 1 : 0;
            const int64_t m0 = static_cast<int64_t>((mt - seg * a.x_tiles) * 2 + rank) * kTile + 32 * quarter, m = m0 + lane;
            // this warp's columns of the tile (a gated pair's features): first .. last - 1
            const int cols = GATED ? a.tile_n / 2 : a.tile_n, first = half * (kTileN / 2), last = min(cols, first + kTileN / 2);
            const int64_t n_tile = static_cast<int64_t>(nt) * cols, end = min(o.R, n_tile + cols);
            // After the CTA's last tile the ring is free: its boxes all have a place of their own there, and no box waits for
            // another's store. fp32 sums that are held in registers, with nothing to follow but a residual, then go to the boxes at once.
            const bool last_tile = tile + tile_step >= a.tiles, f32 = o.y_type == VNM_F32;
            const bool straight = SUM && !GATED && !SPLIT && ALIGNED && last_tile && f32 && o.act == VNM_ACT_NONE && o.bias == nullptr;
            const void* const res = GATED || SPLIT || straight ? nullptr : o.res[seg];  // that the boxes' loop adds
            if (!GATED && !SPLIT && o.res[seg] != nullptr && o.res_vec && m < o.T && n_tile + first < end) {
                // the residual's row is on its way to L2 while the MMAs run
                const int size = f32 ? 4 : 2;
                const uint32_t bytes =
                    static_cast<uint32_t>(min(static_cast<int64_t>(kTileN / 2), end - n_tile - first) * size) & ~15u;
                if (bytes > 0) prefetch_l2(static_cast<const uint8_t*>(o.res[seg]) + (m * o.ld_res + n_tile + first) * size, bytes);
            }
            auto fetch = [&](int c) {  // columns c .. c + 15 of the tile
                Raw16 r;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const Cols at{n_tile + c + 8 * h, end, 1, o.res_vec};
                    if (res != nullptr && m < o.T && !at.none())
                        r.h[h] = load_raw8(res, o.y_type, m * o.ld_res, at);
                    else
                        r.h[h] = Raw8{};
                }
                return r;
            };
            const bool roomy = last_tile && res == nullptr;
            const uint32_t room = smem_base + (warp - kPairHelpers) * (kPairRing / kPairEpilogue);
            const bool bf16 = o.y_type == VNM_BF16, res_tma = res != nullptr && (ALIGNED || o.res_vec);
            const int box_cols = f32 ? 16 : 32;
            // the residual's box from column c on, into output box `at`, whose last store has read it; the outputs then
            // take its place
            auto request = [&](int c, int at) {
                if (!res_tma || m0 >= o.T || n_tile + c >= end) return;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_wait_all_read();
                    const uint32_t bar = smem_u32(&res_bar[GATED ? 0 : warp - kPairHelpers][at & 1]);
                    mbar_arrive_expect_tx(bar, 2048);
                    tma_load_2d(stage + 2048 * (at & 1), &outs.res[seg], static_cast<int32_t>(n_tile + c), static_cast<int32_t>(m0), bar);
                }
                __syncwarp();
                res_pending |= 1u << (at & 1);
            };
            if (!GATED && first < last) request(first, box);
            Scales scale{1.f, 1.f, 1.f, 1.f};
            if constexpr (SUM) {
                // half 0 the first 128 columns of the accumulator, half 1 the others; of a gated pair that is not
                // split, 64 of G's and the same of U's
                float sum[128];
#pragma unroll
                for (int c = 0; c < 128; ++c) sum[c] = 0.f;
                const auto column = [&](int c) { return half * (GATED && !SPLIT ? 64 : 128) + c + (GATED && !SPLIT && c >= 64 ? 64 : 0); };
                for (int kb0 = kb_first; kb0 < kb_last; kb0 += a.chunk_kb) {
                    if (!wait_sum()) break;
                    const uint32_t taddr = tmem + lane_addr + acc * 256;
#pragma unroll
                    for (int c = 0; c < 128; c += LD) {
                        uint32_t v[LD];
                        tmem_ld(taddr + column(c), v);
                        tmem_wait_ld(v);
#pragma unroll
                        for (int j = 0; j < LD; ++j) sum[c + j] += __uint_as_float(v[j]);
                    }
                    if (SPLIT || kb0 + a.chunk_kb < kb_last) release();
                }
                // (the warps that share a barrier below leave there, together)
                if (!run && !(GATED && !SPLIT && o.keep == kKeep8)) break;
                if constexpr (!GATED && !SPLIT && ALIGNED) {
                    if (straight) {
                        release();
                        if (o.res[seg] != nullptr) {
                            // its boxes come all at once to where the outputs' will be, half of them on each barrier
                            const int64_t cols_here = min(static_cast<int64_t>(last), end - n_tile) - first;
                            const int boxes = m0 < o.T && cols_here > 0 ? static_cast<int>(cols_here + 15) / 16 : 0;
                            const uint32_t res_at = smem_u32(&res_bar[GATED ? 0 : warp - kPairHelpers][0]);
                            if (lane == 0 && boxes > 0) {
                                mbar_arrive_expect_tx(res_at, 2048 * min(boxes, 4));
                                if (boxes > 4) mbar_arrive_expect_tx(res_at + 8, 2048 * (boxes - 4));
                                for (int b = 0; b < boxes; ++b)
                                    tma_load_2d(room + 2048 * b, &outs.res[seg], static_cast<int32_t>(n_tile + first + 16 * b),
                                                static_cast<int32_t>(m0), res_at + 8 * (b >> 2));
                            }
                            __syncwarp();
                            res_pending = boxes > 4 ? 3u : boxes > 0 ? 1u : 0u;
#pragma unroll
                            for (int c = 0; c < 128; c += 64) {
                                if (!(res_pending >> (c / 64) & 1u)) break;
                                if (!(run = mbar_wait_warp(res_at + c / 8, res_phase >> (c / 64) & 1u, abort))) break;
                                res_phase ^= 1u << (c / 64);
                                res_pending &= ~(1u << (c / 64));
#pragma unroll
                                for (int u = c; u < c + 64; u += 4) {
                                    // (past the last box: sums that are not stored)
                                    const float4 w = ld_shared_v4(box_piece<64>(room + 2048 * (u / 16), lane, u / 4 % 4));
                                    sum[u] += w.x, sum[u + 1] += w.y, sum[u + 2] += w.z, sum[u + 3] += w.w;
                                }
                            }
                            if (!run) break;
                        }
#pragma unroll
                        for (int c = 0; c < 128; c += 32) {
#pragma unroll
                            for (int u = c; u < c + 32; u += 4)
                                st_shared_f4(box_piece<64>(room + 2048 * (u / 16), lane, u / 4 % 4), sum[u], sum[u + 1], sum[u + 2], sum[u + 3]);
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (first + c < last) {  // (widths are multiples of 32)
                                emit_box<64, 4, true>(&outs.y[seg], true, nullptr, 0, m0, n_tile + first + c, o.T, end, room + 128 * c, lane);
                                emit_box<64, 4, true>(&outs.y[seg], true, nullptr, 0, m0, n_tile + first + c + 16, o.T, end, room + 128 * c + 2048, lane);
                            }
                        }
                        if (lane == 0) tma_store_commit();
                        continue;
                    }
                }
                if constexpr (SPLIT) {
                    // the ring is free: this cluster's MMAs are done with it
                    const int row = 32 * quarter + lane;
#pragma unroll
                    for (int u = 0; u < 32; ++u)
                        st_shared_f4(sum_piece(smem_base, row, 32 * half + u), sum[4 * u], sum[4 * u + 1], sum[4 * u + 2],
                                     sum[4 * u + 3]);
                    fence_proxy_async_smem();
                } else {
                    if constexpr (GATED) {
                        if (o.keep == kKeep8) {
                            // the row's largest magnitudes over the tile's 128 features, a group of the 8-bit
                            // form (features past the edge are zeros): this warp's half and the other's
                            float g = 0.f, u = 0.f;
#pragma unroll
                            for (int c = 0; c < 64; ++c) {
                                g = max_magnitude(g, sum[c]);
                                u = max_magnitude(u, sum[64 + c]);
                            }
                            const uint32_t other = smem_base + kPairRing + ((warp - kPairHelpers) ^ 4) * kStageOut;
                            if (lane == 0) tma_store_wait_all_read();
                            __syncwarp();
                            st_shared_v2(stage + 8 * lane, g, u);
                            // After a wait that ran out in one of the two warps, the sum may still become complete for
                            // the other: both have to leave, or the one that goes on waits here for ever.
                            run = named_barrier_all(1 + quarter, 64, run);
                            if (!run) break;
                            g = max_magnitude(g, ld_shared_f32(other + 8 * lane));
                            u = max_magnitude(u, ld_shared_f32(other + 8 * lane + 4));
                            named_barrier(1 + quarter, 64);  // (read before the boxes are written)
                            scale = scales_of(o, make_float2(g, u), m, nt, half == 0 && m < o.T);
                        }
                    }
                    // back to where the last chunk's sums were, from which the outputs are made as without chunks
                    const uint32_t taddr = tmem + lane_addr + acc * 256;
#pragma unroll
                    for (int c = 0; c < 128; c += 32) {
                        uint32_t v[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(sum[c + j]);
                        tmem_st(taddr + column(c), v);
                    }
                    tmem_wait_st();
                }
            }
            if constexpr (SPLIT) continue;
            uint32_t next[16], next_u[16];
            if constexpr (!GATED) {
                float b[4];  // the bias of columns first + lane, + 32, ...
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t n = n_tile + first + 32 * j + lane;
                    b[j] = o.bias != nullptr && n < end ? load_any(o.bias, o.bias_type, n) : 0.f;
                }
                if (!SUM && !wait_sum()) break;
                const uint32_t taddr = tmem + lane_addr + acc * 256;
                if (first < last) tmem_ld(taddr + first, next);
#pragma unroll 1
                for (int c = first; c < last; c += 16) {
                    float v[16];
                    Raw16 r;  // (a residual of another alignment: by the lanes themselves)
                    if constexpr (!ALIGNED) {
                        if (res != nullptr && !res_tma) r = fetch(c);
                    }
                    tmem_wait_ld(next);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(next[j]);
                    if (c + 16 < last)
                        tmem_ld(taddr + c + 16, next);
                    else
                        release();
                    const int in = c & (box_cols - 1);  // the columns' place in their box
                    const uint32_t buf = roomy ? room + 2048 * ((c - first) / box_cols) : stage + 2048 * (box & 1);
                    const bool landed = res_tma && m0 < o.T && n_tile + c - in < end;
                    if (in == 0) {
                        if (landed) {
                            if (!mbar_wait_warp(smem_u32(&res_bar[GATED ? 0 : warp - kPairHelpers][box & 1]), res_phase >> (box & 1) & 1u, abort)) {
                                run = false;
                                break;
                            }
                            res_phase ^= 1u << (box & 1);
                            res_pending &= ~(1u << (box & 1));
                        } else if (lane == 0 && !roomy) {
                            tma_store_wait_read();
                        }
                        __syncwarp();
                    }
                    if (o.bias != nullptr) {
                        const int k = (c - first) >> 5;
                        const float mine = k == 0 ? b[0] : k == 1 ? b[1] : k == 2 ? b[2] : b[3];
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] += __shfl_sync(0xFFFFFFFFu, mine, ((c - first) & 16) + j);
                    }
                    activate_all(o.act, v);
                    if (landed && f32) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float4 w = ld_shared_v4(box_piece<64>(buf, lane, u));
                            v[4 * u] += w.x, v[4 * u + 1] += w.y, v[4 * u + 2] += w.z, v[4 * u + 3] += w.w;
                        }
                    } else if (landed || (!ALIGNED && res != nullptr && !res_tma)) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float w[8];
                            if (ALIGNED || landed) {
                                const float4 q = ld_shared_v4(box_piece<64>(buf, lane, in / 8 + h));
                                widen8(make_uint4(__float_as_uint(q.x), __float_as_uint(q.y), __float_as_uint(q.z), __float_as_uint(q.w)),
                                       bf16, w);
                            } else {
                                widen_raw8(r.h[h], o.y_type, w);
                            }
#pragma unroll
                            for (int j = 0; j < 8; ++j) v[8 * h + j] += w[j];
                        }
                    }
                    if (f32) {
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            st_shared_f4(box_piece<64>(buf, lane, u), v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
                    } else {
                        uint32_t w[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u) w[u] = bf16 ? to_bf16x2(v[2 * u], v[2 * u + 1]) : to_f16x2(v[2 * u], v[2 * u + 1]);
                        st_shared_v4(box_piece<64>(buf, lane, in / 8), w[0], w[1], w[2], w[3]);
                        st_shared_v4(box_piece<64>(buf, lane, in / 8 + 1), w[4], w[5], w[6], w[7]);
                    }
                    // (at the box's end, so that the last box's store has read the other one)
                    if (in == box_cols - 16 && c + 16 < last) request(c + 16, box + 1);
                    if (in + 16 < box_cols) continue;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (f32)
                        emit_box<64, 4, ALIGNED>(&outs.y[seg], o.y_tma, o.y[seg], o.ld_y, m0, n_tile + c, o.T, end, buf, lane);
                    else
                        emit_box<64, 2, ALIGNED>(&outs.y[seg], o.y_tma, o.y[seg], o.ld_y, m0, n_tile + c - 16, o.T, end, buf, lane);
                    if (lane == 0) tma_store_commit();
                    ++box;
                }
            } else {
                if (!SUM && !wait_sum()) break;
                const uint32_t taddr = tmem + lane_addr + acc * 256;
                if (first < last) {
                    tmem_ld(taddr + first, next);
                    tmem_ld(taddr + cols + first, next_u);
                }
                const bool twice = o.keep == kKeepNone;  // two boxes
                const int box_cols = o.keep == kKeep16 ? 16 : 32;
#pragma unroll 1
                for (int c = first; c < last; c += 16) {
                    float g[16], u[16];
                    tmem_wait_ld(next);
                    tmem_wait_ld(next_u);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        g[j] = __uint_as_float(next[j]);
                        u[j] = __uint_as_float(next_u[j]);
                    }
                    if (c + 16 < last) {
                        tmem_ld(taddr + c + 16, next);
                        tmem_ld(taddr + cols + c + 16, next_u);
                    } else {
                        release();
                    }
                    const int in = c & (box_cols - 1);
                    const uint32_t buf = roomy ? room + 4096 * ((c - first) / box_cols) : stage + (twice ? 2048 * (box & 1) : 0);
                    if (in == 0) {
                        if (lane == 0 && !roomy) {
                            if (twice)
                                tma_store_wait_read();
                            else
                                tma_store_wait_all_read();
                        }
                        __syncwarp();
                    }
                    auto pack16 = [&](const float (&v)[16], uint32_t (&w)[8]) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) w[j] = bf16 ? to_bf16x2(v[2 * j], v[2 * j + 1]) : to_f16x2(v[2 * j], v[2 * j + 1]);
                    };
                    auto stage16 = [&](uint32_t to, const float (&v)[16]) {  // rows of 32 bytes
                        uint32_t w[8];
                        pack16(v, w);
                        st_shared_v4(box_piece<32>(to, lane, 0), w[0], w[1], w[2], w[3]);
                        st_shared_v4(box_piece<32>(to, lane, 1), w[4], w[5], w[6], w[7]);
                    };
                    auto stage8 = [&](uint32_t to, const float (&v)[16], float s, float inv) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = to_fp8x4(quotient(v[4 * j], s, inv), quotient(v[4 * j + 1], s, inv),
                                            quotient(v[4 * j + 2], s, inv), quotient(v[4 * j + 3], s, inv), o.e5m2);
                        st_shared_v4(box_piece<32>(to, lane, in / 16), w[0], w[1], w[2], w[3]);
                    };
                    if (o.keep == kKeep16) {
                        stage16(buf + 1024, g);
                        stage16(buf + 2048, u);
                    } else if (o.keep == kKeep8) {
                        stage8(buf + 2048, g, scale.g, scale.g_inv);
                        stage8(buf + 3 * 1024, u, scale.u, scale.u_inv);
                    }
                    activate_all(o.act, g);
#pragma unroll
                    for (int j = 0; j < 16; ++j) g[j] *= u[j];
                    if (o.keep == kKeep16) {
                        stage16(buf, g);
                    } else {
                        uint32_t w[8];
                        pack16(g, w);
                        st_shared_v4(box_piece<64>(buf, lane, in / 8), w[0], w[1], w[2], w[3]);
                        st_shared_v4(box_piece<64>(buf, lane, in / 8 + 1), w[4], w[5], w[6], w[7]);
                    }
                    if (in + 16 < box_cols) continue;
                    fence_proxy_async_smem();
                    __syncwarp();
                    const int64_t n0 = n_tile + c - in;
                    if (o.keep == kKeep16) {
                        emit_box<32, 2, ALIGNED>(&outs.y[0], o.y_tma, o.y[0], o.ld_y, m0, n0, o.T, end, buf, lane);
                        emit_box<32, 2, ALIGNED>(&outs.g, o.keep_tma, o.g.p, o.g.ld, m0, n0, o.T, end, buf + 1024, lane);
                        emit_box<32, 2, ALIGNED>(&outs.u, o.keep_tma, o.u.p, o.u.ld, m0, n0, o.T, end, buf + 2048, lane);
                    } else {
                        emit_box<64, 2, ALIGNED>(&outs.y[0], o.y_tma, o.y[0], o.ld_y, m0, n0, o.T, end, buf, lane);
                    }
                    if (o.keep == kKeep8) {
                        emit_box<32, 1, ALIGNED>(&outs.g, o.keep_tma, o.g.p, o.g.ld, m0, n0, o.T, end, buf + 2048, lane);
                        emit_box<32, 1, ALIGNED>(&outs.u, o.keep_tma, o.u.p, o.u.ld, m0, n0, o.T, end, buf + 3 * 1024, lane);
                    }
                    if (lane == 0) tma_store_commit();
                    ++box;
                }
            }
            if (first >= last) release();
        }
        if (lane == 0) tma_store_wait_all_read();
        for (int at = 0; at < 2; ++at)  // (after a wait that ran out) copies in flight must land before the CTA exits
            if (res_pending >> at & 1u) mbar_drain(smem_u32(&res_bar[GATED ? 0 : warp - kPairHelpers][at]), res_phase >> at & 1u);
    }

    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();  // no CTA leaves while the others' arrivals, MMAs or reads may reach it
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_group<2>(tmem, 512);
    }
    if constexpr (SPLIT) {
        // Add the pairs' sums, in their order, each pair a share of the rows: every CTA copies the other shares to their
        // owners, behind the owners' own sums (reading them there instead, 16 bytes a lane, took 7 us).
        const OutArgs& o = a.o;
        const bool vec = all_vec(o);
        const int share = (kTile + a.splits - 1) / a.splits, row0 = pair * share, row1 = min(kTile, row0 + share);
        const uint32_t bar = smem_u32(&split_bar), landing = smem_base + kSumBytes;
        if (threadIdx.x == 0) {
            mbar_arrive_expect_tx(bar, static_cast<uint32_t>((a.splits - 1) * (row1 - row0) * 1024));
            for (int p = 0; p < a.splits; ++p) {
                if (p == pair) continue;
                const int first = p * share, rows = min(kTile, first + share) - first, slot = pair < p ? pair : pair - 1;
                copy_to_cluster(dsmem_map(landing + slot * share * 1024, 2 * p + rank), smem_base + first * 1024,
                                static_cast<uint32_t>(rows * 1024), dsmem_map(bar, 2 * p + rank));
            }
        }
        int mt, nt;
        tile_at(a, tile0, mt, nt);
        const int seg = a.kind == kTwoByRows && mt >= a.x_tiles ? 1 : 0;
        const int64_t m0 = static_cast<int64_t>((mt - seg * a.x_tiles) * 2 + rank) * kTile;
        constexpr int kLanes = GATED ? 16 : 32, kRowsAtOnce = 32 / kLanes;  // of a row
        const int q = lane & (kLanes - 1);
        const int local = vec ? 8 * q : q, step = vec ? 1 : kLanes;
        const Cols c{static_cast<int64_t>(nt) * kTileN + local, o.R, step, vec};
        float b[8];
        bias8(o, c, b);
        const bool landed = mbar_wait_warp(bar, 0, abort);
        if (!landed) mbar_drain(bar, 0);  // (after a wait that ran out) no CTA leaves while the others' sums are on their way to it
#pragma unroll 1
        for (int base = row0 + kRowsAtOnce * warp; base < row1 && landed; base += kRowsAtOnce * (kPairThreads / 32)) {
            const int row = min(base + lane / kLanes, row1 - 1);
            const int64_t t = m0 + row;
            const bool here = base + lane / kLanes < row1 && t < o.T;
            float v[GATED ? 2 : 1][8];
            Raw8 r;
            if (!GATED && here && o.res[seg] != nullptr && !c.none()) r = load_raw8(o.res[seg], o.y_type, t * o.ld_res, c);
#pragma unroll
            for (int h = 0; h < (GATED ? 2 : 1); ++h) {
                const int col = 128 * h + local;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[h][j] = 0.f;
#pragma unroll
                for (int s = 0; s < kMaxPairSplits; ++s) {
                    if (s >= a.splits) break;
                    // (the pieces keep the order that row & 7 gave them)
                    const uint32_t from = s == pair ? smem_base : landing + ((s < pair ? s : s - 1) * share - row0) * 1024;
                    if (vec) {
                        const float4 x = ld_shared_v4(sum_piece(from, row, col >> 2)), y = ld_shared_v4(sum_piece(from, row, (col >> 2) + 1));
                        v[h][0] += x.x, v[h][1] += x.y, v[h][2] += x.z, v[h][3] += x.w;
                        v[h][4] += y.x, v[h][5] += y.y, v[h][6] += y.z, v[h][7] += y.w;
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[h][j] += ld_shared_f32(sum_at(from, row, col + step * j));
                    }
                }
            }
            if constexpr (GATED) {
                Scales s{1.f, 1.f, 1.f, 1.f};
                if (o.keep == kKeep8) s = scales_of(o, largest_of<16>(v[0], v[1]), t, nt, here && q == 0);
                if (here && !c.none()) {
                    keep_gated8(o, t, c, v[0], v[1], s);
                    finish_gated8(o, t, c, v[0], v[1]);
                }
            } else if (here) {
                finish8(o, seg, t, c, v[0], b, r);
            }
        }
        cluster_sync_all();  // no CTA leaves while its sums are copied from it
    }
    if (a.beside) after_previous_grid();
    if (threadIdx.x == 0 && abort_flag) record_error(a.status ? a.status : g_status, VNM_ERR_TIMEOUT, 13);
}

// ------------------------------------------------------------------ narrow tiles

// Of a gated pair a tile's 128 rows are 64 of Wg's and the same 64 of Wu's.
template <int BN>
struct NarrowCfg {
    static constexpr int kStageBytes = kOperandBytes + BN * 128;
    static constexpr int kStages = BN == 128 ? 3 : BN == 64 ? 4 : 5;
    static constexpr int kTmemCols = 2 * BN;  // two chunks' sums
    static constexpr int kThreads = 192;
    static constexpr int kSmem = kStages * kStageBytes + 1024;
    static_assert(kTile * BN * 4 <= kStages * kStageBytes, "the CTA's sums fit the stage ring");
    // two CTAs an SM, whose waits overlap
    static_assert(2 * (kSmem + 4096) <= 228 * 1024 && 2 * kTmemCols <= 512 && kTmemCols >= 32, "shared memory and TMEM of two CTAs");
};

template <int BN, bool GATED>
__global__ void __launch_bounds__(NarrowCfg<BN>::kThreads, 2)
    dense_narrow_kernel(const __grid_constant__ Maps maps, const __grid_constant__ GemmArgs a) {
    using Cfg = NarrowCfg<BN>;
    constexpr int ST = Cfg::kStages;
    constexpr int kFeatures = GATED ? 64 : 128;  // columns of Y of a tile
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[ST], empty_bar[ST];
    __shared__ __align__(8) uint64_t accf_bar[2], acce_bar[2];
    __shared__ float2 tops[GATED ? BN : 1];  // of each token: G's and U's largest magnitudes over the tile
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    float* const part = reinterpret_cast<float*>(smem_raw + (smem_base - smem_u32(smem_raw)));  // [BN][kTile], over the ring
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // CTAs of a cluster: the splits of a tile, or (8-bit checkpoints) of two tiles, which share a group's 128 features
    const bool twin = GATED && a.o.keep == kKeep8;
    const int rank = static_cast<int>(blockIdx.x) % a.splits;
    int mt, nt;  // tiles of W's rows and of tokens; those fastest: the CTAs that run together share W's tiles
    if (twin) {
        const int two = static_cast<int>(blockIdx.x) / (2 * a.splits);
        mt = 2 * (two / a.n_tiles) + static_cast<int>(blockIdx.x) / a.splits % 2;
        nt = two % a.n_tiles;
    } else {
        const int tile = static_cast<int>(blockIdx.x) / a.splits;
        mt = tile / a.n_tiles;
        nt = tile % a.n_tiles;
    }
    const int seg = a.kind == kTwoByRows && nt >= a.x_tiles ? 1 : 0;
    const int xrow = (nt - seg * a.x_tiles) * BN, wrow = mt * kFeatures;
    const int kb0 = min(a.total_kb, rank * a.kb_per_split), kb1 = min(a.total_kb, kb0 + a.kb_per_split);

    // one stage's loads into its slot
    auto load_stage = [&](int slot, int kb) {
        const uint32_t fb = smem_u32(&full_bar[slot]), sw = smem_base + slot * Cfg::kStageBytes, sx = sw + kOperandBytes;
        const bool second = kb >= a.num_kb;  // of a sum of two
        const CUtensorMap *tx = &maps.x[second || seg], *tw = &maps.w[second];
        const int k = (second ? kb - a.num_kb : kb) * kBlockK;
        mbar_arrive_expect_tx(fb, Cfg::kStageBytes);
        if (GATED) {
            tma_load_2d(sw, &maps.w[0], k, wrow, fb);
            tma_load_2d(sw + 8192, &maps.w[1], k, wrow, fb);
        } else if (a.w_t) {
            tma_load_2d(sw, tw, wrow, k, fb);
            tma_load_2d(sw + 8192, tw, wrow + 64, k, fb);
        } else {
            tma_load_2d(sw, tw, k, wrow, fb);
        }
        if (a.x_t) {  // (tiles of 64 or 128 tokens only)
            tma_load_2d(sx, tx, xrow, k, fb);
            if (BN == 128) tma_load_2d(sx + 8192, tx, xrow + 64, k, fb);
        } else {
            tma_load_2d(sx, tx, k, xrow, fb);
        }
    };
    const int early = min(ST, kb1 - kb0);  // stages loaded before the setup is over
    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(smem_u32(&full_bar[s]), 1);
            mbar_init(smem_u32(&empty_bar[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&accf_bar[s]), 1);
            mbar_init(smem_u32(&acce_bar[s]), 4);
        }
        abort_flag = 0;
        fence_barrier_init();
        // the first stages need no other thread: their latency covers the TMEM allocation
        after_the_one_before(a.beside, false);
        for (int k = 0; k < early; ++k)
            if (k != a.skip_stage || blockIdx.x != 0) load_stage(k, kb0 + k);
    }
    if (warp == 1) tmem_alloc_group<1>(smem_u32(&tmem_slot), Cfg::kTmemCols);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    after_the_one_before(a.beside, a.o.res[0] != nullptr);
    if (a.next_beside) let_next_grid_start();
    const uint32_t tmem = tmem_slot;
    volatile int* abort = &abort_flag;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        int it = early;
        for (; it < kb1 - kb0; ++it) {
            const int slot = it % ST;
            if (!mbar_wait_warp(smem_u32(&empty_bar[slot]), (static_cast<uint32_t>(it / ST) & 1u) ^ 1u, abort)) break;
            if (elect_one() && (it != a.skip_stage || blockIdx.x != 0)) load_stage(slot, kb0 + it);
            __syncwarp();
        }
        if (*abort)  // every copy issued must land before the CTA exits
            for (int k = it > ST ? it - ST : 0; k < it; ++k)
                if (k != a.skip_stage || blockIdx.x != 0)
                    mbar_drain(smem_u32(&full_bar[k % ST]), static_cast<uint32_t>(k / ST) & 1u);
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        const uint64_t wdesc = operand_desc(smem_base, a.w_t), xdesc = operand_desc(smem_base + kOperandBytes, a.x_t);
        const uint32_t wstep = operand_step(a.w_t), xstep = operand_step(a.x_t);
        int it = 0, slot = 0, chunk = 0;
        uint32_t phase = 0;
        bool run = true;
        for (int c0 = kb0; c0 < kb1 && run; c0 += a.chunk_kb, ++chunk) {
            const int c1 = min(kb1, c0 + a.chunk_kb), acc = chunk & 1;
            if (chunk >= 2 && !mbar_wait_warp(smem_u32(&acce_bar[acc]), (static_cast<uint32_t>(chunk >> 1) & 1u) ^ 1u, abort)) break;
            for (int kb = c0; kb < c1; ++kb, ++it) {
                if (!mbar_wait_warp(smem_u32(&full_bar[slot]), phase, abort)) {
                    run = false;
                    break;
                }
                tc_fence_after_sync();
                if (elect_one()) {
                    const uint64_t off = static_cast<uint64_t>((slot * Cfg::kStageBytes) >> 4);
#pragma unroll
                    for (uint32_t s = 0; s < 4; ++s)
                        tc_mma_f16(tmem + acc * BN, wdesc + off + s * wstep, xdesc + off + s * xstep, a.idesc,
                                   kb > c0 || s > 0 ? 1u : 0u);
                    tc_commit(smem_u32(&empty_bar[slot]));
                    if (kb + 1 == c1) tc_commit(smem_u32(&accf_bar[acc]));
                }
                __syncwarp();
                if (++slot == ST) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
        // every MMA issued is done before TMEM goes back
        if (it > 0) mbar_drain(smem_u32(&empty_bar[(it - 1) % ST]), static_cast<uint32_t>((it - 1) / ST) & 1u);
    } else {
        // ------------------------------------------------ the CTA's sums to shared memory
        const int quarter = warp & 3, row = 32 * quarter + lane;
        const uint32_t lane_addr = static_cast<uint32_t>(32 * quarter) << 16;
        constexpr int LD = BN >= 32 ? 32 : 16;
        float sum[BN];
#pragma unroll
        for (int c = 0; c < BN; ++c) sum[c] = 0.f;
        bool run = true;
        int chunk = 0;
        for (int c0 = kb0; c0 < kb1; c0 += a.chunk_kb, ++chunk) {
            const int acc = chunk & 1;
            if (!(run = mbar_wait_warp(smem_u32(&accf_bar[acc]), static_cast<uint32_t>(chunk >> 1) & 1u, abort))) break;
            tc_fence_after_sync();
#pragma unroll
            for (int c = 0; c < BN; c += LD) {
                uint32_t v[LD];
                tmem_ld(tmem + lane_addr + acc * BN + c, v);
                tmem_wait_ld(v);
#pragma unroll
                for (int j = 0; j < LD; ++j) sum[c + j] += __uint_as_float(v[j]);
            }
            tc_fence_before_sync();
            __syncwarp();
            if (elect_one()) mbar_arrive(smem_u32(&acce_bar[acc]));
        }
        // the ring is free: the MMAs of the last chunk are done with it
        if (run) {
#pragma unroll
            for (int c = 0; c < BN; ++c) part[c * kTile + row] = sum[c];
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    let_next_grid_start();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_group<1>(tmem, Cfg::kTmemCols);
    }
    if (a.splits > 1) cluster_sync_all();
    // add the cluster's sums, in rank order, each CTA a share of the tokens; kLanes lanes x 8 columns a token
    constexpr int kLanes = kFeatures / 8, kAtOnce = 32 / kLanes, kStep = kAtOnce * (Cfg::kThreads / 32);
    const int share = (BN + a.splits - 1) / a.splits, first = rank * share, last = min(BN, first + share);
    const int tile_rank = (twin && (mt & 1) ? a.splits : 0);  // the tile's first CTA in the cluster
    const OutArgs& o = a.o;
    const bool vec = all_vec(o);
    const int q = lane & (kLanes - 1), local = vec ? 8 * q : q, step = vec ? 1 : kLanes;
    const Cols cols{static_cast<int64_t>(wrow) + local, o.R, step, vec};
    float bias[8];
    bias8(o, cols, bias);
    // the sums of token c of the tile at the lane's columns, from row `row0` of the tile on
    auto gather = [&](int c, int row0, float (&v)[8]) {
        const uint32_t addr = smem_base + 4 * (min(c, BN - 1) * kTile + row0 + local);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
        if (a.splits == 1) {  // (this CTA's own)
            if (vec) {
                const float4 x = ld_shared_v4(addr), y = ld_shared_v4(addr + 16);
                v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
                v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = ld_shared_f32(addr + 4 * kLanes * j);
            }
            return;
        }
#pragma unroll
        for (int s = 0; s < kMaxSplits; ++s) {
            if (s >= a.splits) break;
            const uint32_t from = dsmem_map(addr, tile_rank + s);
            if (vec) {
                const float4 x = dsmem_ld_v4(from), y = dsmem_ld_v4(from + 16);
                v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
                v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += dsmem_ld_f32(from + 4 * kLanes * j);
            }
        }
    };
    if constexpr (GATED) {
        if (twin) {
            // (features past the edge are zeros)
#pragma unroll 1
            for (int base = first + kAtOnce * warp; base < last; base += kStep) {
                const int c = base + lane / kLanes;
                float g[8], u[8];
                gather(c, 0, g);
                gather(c, 64, u);
                const float2 m = largest_of<kLanes>(g, u);
                if (c < last && q == 0) tops[c] = m;
            }
            cluster_sync_all();
        }
    }
#pragma unroll 1
    for (int base = first + kAtOnce * warp; base < last; base += kStep) {
        const int c = base + lane / kLanes;
        const int64_t t = static_cast<int64_t>(xrow) + c;
        const bool here = c < last && t < o.T;
        float v[8];
        if constexpr (GATED) {
            float u[8];
            gather(c, 0, v);
            gather(c, 64, u);
            Scales s{1.f, 1.f, 1.f, 1.f};
            if (twin) {
                const int at = min(c, BN - 1);
                // the other tile's CTA of the same rank
                const uint32_t other = dsmem_map(smem_u32(&tops[at]), (mt & 1 ? 0 : a.splits) + rank);
                const float2 m = make_float2(max_magnitude(tops[at].x, dsmem_ld_f32(other)),
                                             max_magnitude(tops[at].y, dsmem_ld_f32(other + 4)));
                s = scales_of(o, m, t, mt >> 1, here && q == 0 && (mt & 1) == 0);
            }
            if (here && !cols.none()) {
                keep_gated8(o, t, cols, v, u, s);
                finish_gated8(o, t, cols, v, u);
            }
        } else {
            Raw8 r;
            if (here && o.res[seg] != nullptr && !cols.none()) r = load_raw8(o.res[seg], o.y_type, t * o.ld_res, cols);
            gather(c, 0, v);
            if (here) finish8(o, seg, t, cols, v, bias, r);
        }
    }
    if (a.splits > 1 || twin) cluster_sync_all();  // no CTA leaves while others read its sums
    if (a.beside) after_previous_grid();
    if (threadIdx.x == 0 && abort_flag) record_error(a.status ? a.status : g_status, VNM_ERR_TIMEOUT, 14);
}

// K = 0: the sums are 0.
__global__ void dense_empty_kernel(const OutArgs o, int kind) {
    after_previous_grid();
    const int64_t per_row = (o.R + 7) / 8;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < o.T * per_row;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t t = i / per_row;
        const Cols c{8 * (i - t * per_row), o.R, 1, all_vec(o)};
        float v[8] = {}, u[8] = {}, b[8];
        if (kind == kGatedPair) {
            if (o.keep == kKeep8 && c.first % 128 == 0) {
                o.g.s[t * o.g.s_rs + (c.first / 128) * o.g.s_cs] = kMinScale;
                o.u.s[t * o.u.s_rs + (c.first / 128) * o.u.s_cs] = kMinScale;
            }
            keep_gated8(o, t, c, v, u, Scales{kMinScale, 1.f / kMinScale, kMinScale, 1.f / kMinScale});
            finish_gated8(o, t, c, v, u);
            continue;
        }
        bias8(o, c, b);
        for (int seg = 0; seg < (kind == kTwoByRows ? 2 : 1); ++seg) {
            float w[8] = {};
            Raw8 r;
            if (o.res[seg] != nullptr) r = load_raw8(o.res[seg], o.y_type, t * o.ld_res, c);
            finish8(o, seg, t, c, w, b, r);
        }
    }
}

// ------------------------------------------------------------------ host side

int64_t ceil_div(int64_t p, int64_t q) { return (p + q - 1) / q; }

// An operand (rows x K) as boxes of 64 elements of K by `box_rows` rows; transposed, of 64 rows by 64 of K.
bool encode(CUtensorMap* tm, const Operand16& x, int64_t rows, int64_t K, bool bf16, int box_rows) {
    const CUtensorMapDataType t = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return x.transposed ? encode_2d(tm, t, x.p, rows, K, x.ld * 2, 64, kBlockK, CU_TENSOR_MAP_SWIZZLE_128B)
                        : encode_2d(tm, t, x.p, K, rows, x.ld * 2, kBlockK, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool encode_all(Maps* m, const ProductArgs& p, int x_rows, int w_rows) {
    const int nx = p.kind == kSumOfTwo || p.kind == kTwoByRows ? 2 : 1, nw = p.kind == kSumOfTwo || p.kind == kGatedPair ? 2 : 1;
    for (int i = 0; i < 2; ++i)
        if (!encode(&m->x[i], p.x[std::min(i, nx - 1)], p.T, p.K, p.bf16, x_rows) ||
            !encode(&m->w[i], p.w[std::min(i, nw - 1)], p.R, p.K, p.bf16, w_rows))
            return false;
    return true;
}

// The outputs, and residuals, that go by tensor memory copies, as boxes of 32 rows; the others' maps are not used.
bool encode_outputs(OutMaps* m, const ProductArgs& p, const OutArgs& o) {
    auto type = [](vnm_dtype t) {
        return t == VNM_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
               : t == VNM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                              : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    };
    const bool gated = p.kind == kGatedPair, eight = p.keep == kKeep8, sixteen = p.keep == kKeep16;
    const int e = p.y_type == VNM_F32 ? 4 : 2, wide = sixteen ? 16 : 64 / e;  // columns of a box of Y
    *m = OutMaps{};
    if (o.y_tma)
        for (int i = 0; i < (p.kind == kTwoByRows ? 2 : 1); ++i)
            if (!encode_2d(&m->y[i], type(p.y_type), p.y[i], p.R, p.T, p.ld_y * e, wide, 32,
                           sixteen ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B))
                return false;
    if (!gated && p.residual[0] != nullptr && o.res_vec)
        for (int i = 0; i < (p.kind == kTwoByRows ? 2 : 1); ++i)
            if (!encode_2d(&m->res[i], type(p.y_type), p.residual[i], p.R, p.T, p.ld_residual * e, wide, 32, CU_TENSOR_MAP_SWIZZLE_64B))
                return false;
    if (!o.keep_tma) return true;
    const CUtensorMapDataType t = eight ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : type(p.y_type);
    const int bytes = eight ? 1 : 2;
    return encode_2d(&m->g, t, p.g.p, p.R, p.T, p.g.ld * bytes, 32 / bytes, 32, CU_TENSOR_MAP_SWIZZLE_32B) &&
           encode_2d(&m->u, t, p.u.p, p.R, p.T, p.u.ld * bytes, 32 / bytes, 32, CU_TENSOR_MAP_SWIZZLE_32B);
}

template <typename Kernel>
cudaError_t prepare(Kernel kernel, int smem, int regs, std::atomic<bool>* set) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevicesDl) return cudaErrorInvalidDevice;
    if (set[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    if (regs > 0) {
        // the shares are drawn from the launch's registers: never ask for more
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, kernel)) != cudaSuccess) return e;
        if (fa.numRegs != regs) return cudaErrorInvalidConfiguration;
    }
    set[dev].store(true, std::memory_order_relaxed);
    return cudaSuccess;
}

template <bool GATED, bool SUM, bool SPLIT, bool ALIGNED>
cudaError_t run_pair(const ProductArgs& p, GemmArgs a, int tile_n, int splits, int sm_count, cudaStream_t stream) {
    static std::atomic<bool> set[kMaxDevicesDl];
    a.x_tiles = static_cast<int>(ceil_div(p.T, 2 * kTile));
    a.m_tiles = a.x_tiles * (p.kind == kTwoByRows ? 2 : 1);
    a.n_tiles = static_cast<int>(ceil_div(p.R, GATED ? tile_n / 2 : tile_n));
    a.tile_n = tile_n;
    // (transposed W comes in boxes of 64 rows)
    a.stage_bytes = kOperandBytes + (a.w_t ? static_cast<int>(ceil_div(tile_n, 128)) * 8192 : tile_n / 2 * 128);
    a.stages = std::min(kPairMaxStages, kPairRing / a.stage_bytes);
    const int64_t tiles = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    a.tiles = static_cast<int>(tiles);
    if (tiles * 2 * splits > INT32_MAX) return cudaErrorInvalidValue;
    a.splits = splits;
    a.kb_per_split = static_cast<int>(ceil_div(a.total_kb, splits));
    a.idesc = f16_idesc(2 * kTile, tile_n, p.bf16, a.x_t, a.w_t);
    Maps maps;
    OutMaps outs;
    if (!encode_all(&maps, p, kTile, tile_n / 2) || (!SPLIT && !encode_outputs(&outs, p, a.o))) return cudaErrorInvalidValue;
    const auto kernel = dense_pair_kernel<GATED, SUM, SPLIT, ALIGNED>;
    const cudaError_t e = prepare(kernel, kPairSmem, SUM && !SPLIT ? kSumLaunchRegs : 0, set);
    if (e != cudaSuccess) return e;
    const int64_t pairs = SPLIT ? tiles * splits : std::min<int64_t>(tiles, std::max(1, sm_count / 2));
    return launch_early(kernel, 2 * pairs, kPairThreads, kPairSmem, 2 * splits, stream, maps, outs, a);
}

template <bool GATED>
cudaError_t run_pair(const ProductArgs& p, const GemmArgs& a, bool sum, bool aligned, int tile_n, int sm_count, cudaStream_t stream) {
    if (sum)
        return aligned ? run_pair<GATED, true, false, true>(p, a, tile_n, 1, sm_count, stream)
                       : run_pair<GATED, true, false, false>(p, a, tile_n, 1, sm_count, stream);
    return aligned ? run_pair<GATED, false, false, true>(p, a, tile_n, 1, sm_count, stream)
                   : run_pair<GATED, false, false, false>(p, a, tile_n, 1, sm_count, stream);
}

template <int BN, bool GATED>
cudaError_t run_narrow(const ProductArgs& p, GemmArgs a, int splits, cudaStream_t stream) {
    using Cfg = NarrowCfg<BN>;
    static std::atomic<bool> set[kMaxDevicesDl];
    const int twin = p.keep == kKeep8 ? 2 : 1;
    a.x_tiles = static_cast<int>(ceil_div(p.T, BN));
    a.n_tiles = a.x_tiles * (p.kind == kTwoByRows ? 2 : 1);
    a.m_tiles = static_cast<int>(ceil_div(p.R, GATED ? 64 * twin : kTile)) * twin;
    const int64_t tiles = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
    if (tiles * splits > INT32_MAX) return cudaErrorInvalidValue;
    a.tiles = static_cast<int>(tiles);
    a.splits = splits;
    a.kb_per_split = static_cast<int>(ceil_div(a.total_kb, splits));
    a.idesc = f16_idesc(kTile, BN, p.bf16, a.w_t, a.x_t);
    Maps maps;
    if (!encode_all(&maps, p, BN, GATED ? 64 : kTile)) return cudaErrorInvalidValue;
    const cudaError_t e = prepare(dense_narrow_kernel<BN, GATED>, Cfg::kSmem, 0, set);
    if (e != cudaSuccess) return e;
    return launch_early(dense_narrow_kernel<BN, GATED>, tiles * splits, Cfg::kThreads, Cfg::kSmem, splits * twin, stream, maps, a);
}

template <bool GATED>
cudaError_t run_narrow(int bn, const ProductArgs& p, const GemmArgs& a, int splits, cudaStream_t stream) {
    switch (bn) {
        case 16: return run_narrow<16, GATED>(p, a, splits, stream);
        case 32: return run_narrow<32, GATED>(p, a, splits, stream);
        case 64: return run_narrow<64, GATED>(p, a, splits, stream);
        default: return run_narrow<128, GATED>(p, a, splits, stream);
    }
}

// The times that the plan compares, in us. The constants were fitted to 218 products of random sizes (T = 9 .. 8192,
// R = 64 .. 11008, K = 64 .. 11008, all operand orders, checkpoints or none), each timed with every plan that there was: pairs
// of 256, 192 and 128 columns, all splits, all narrow tiles. What the rule picked was 1.6 % slower than the fastest on average,
// 25 % at worst; for 219 other such products 2.2 %, a few 30 %, one (which now takes another plan) 82 %. Pairs of 160 and 224
// columns came later; eleven products were timed with them, where they win by 6 % at most. The constants weigh the plans against
// each other; the absolute times are up to a third off. `aligned` is about the starts of Y's rows and of an 8-bit G's: rows that
// end inside 16 bytes, and a residual, U or 16-bit checkpoint off 16 bytes, take the other variant too, which the times leave out.
TilePlan plan_tiles(const ProductArgs& p, int sm_count) {
    const bool gated = p.kind == kGatedPair, two = p.kind == kTwoByRows, keep8 = p.keep == kKeep8;
    const int64_t e = p.y_type == VNM_F32 ? 4 : 2;
    const bool aligned = (reinterpret_cast<uintptr_t>(p.y[0]) | static_cast<uintptr_t>(p.ld_y * e)) % 16 == 0 &&
                         (!keep8 || (reinterpret_cast<uintptr_t>(p.g.p) | static_cast<uintptr_t>(p.g.ld)) % 16 == 0);
    const int64_t num_kb = ceil_div(p.K, kBlockK) * (p.kind == kSumOfTwo ? 2 : 1);
    TilePlan best{0, 1, 256};
    double least = 1e30;
    auto consider = [&](const TilePlan& plan, double t) {
        if (t < least) {
            least = t;
            best = plan;
        }
    };
    // Pairs of CTAs. A K block takes the MMAs' time, or what the running pairs load from L2 (10.3 TB/s) or the
    // tiles' own rows of W from memory (5.3 TB/s) takes; a tile's epilogue runs under the next one's K blocks.
    constexpr double kSetup = 5.5, kMma = 0.43, kLeast = 0.32, kL2 = 10.3e6, kMemory = 5.3e6;
    const int64_t row_tiles = ceil_div(p.T, 2 * kTile) * (two ? 2 : 1), pairs = std::max(1, sm_count / 2);
    for (int n = 256; n >= 128; n -= gated ? 64 : 32) {  // (boxes of 32 columns or features)
        // (a group of the 8-bit form is 128 features; a warp that adds chunks up holds 64 of both products)
        if (n < 256 && gated && (keep8 || num_kb > kLongChunk)) break;
        const int64_t tiles = row_tiles * ceil_div(p.R, gated ? n / 2 : n), full = tiles / pairs, rest = tiles % pairs;
        const double epilogue = (gated ? (keep8 ? 1.4 : 0.0) + (aligned ? 0.0 : 1.1) : aligned ? 0.9 : 6.0) * n / 256;
        auto block = [&](int64_t active) {
            return std::max(std::max(kMma * n / 256, kLeast),
                            std::max(static_cast<double>(2 * active * (kOperandBytes + 64 * n)) / kL2,
                                     static_cast<double>(active * n * 128) / static_cast<double>(row_tiles) / kMemory));
        };
        double t = kSetup + epilogue + static_cast<double>(full) * std::max(num_kb * block(pairs), epilogue);
        if (rest > 0) t += std::max(num_kb * block(rest), full > 0 ? epilogue : 0.0);
        consider({0, 1, n}, t);
    }
    // K over the pairs of a cluster: as many clusters as fit at once (of 4, 6 and 8 CTAs, one an SM).
    const int64_t pair_tiles = row_tiles * ceil_div(p.R, gated ? 128 : 256);
    for (int splits = 2; splits <= kMaxPairSplits && splits <= num_kb; ++splits) {
        const int64_t clusters = std::max(1, sm_count * (splits == 2 ? 36 : splits == 3 ? 23 : 15) / 152);
        consider({0, splits, 256}, kSetup + static_cast<double>(ceil_div(pair_tiles, clusters)) *
                                                (static_cast<double>(ceil_div(num_kb, splits)) * kMma + 4.5));
    }
    // Narrow tiles, two CTAs an SM: a launch, a wave's chain of K blocks (longer where SMs run two CTAs, or as long as
    // the loads from L2 take), its end; or the operands from memory.
    const double memory = 2.0 * static_cast<double>(p.K) * static_cast<double>((gated ? 2 : 1) * p.R + p.T) / kMemory;
    for (int i = 0; i < 4; ++i) {
        const int bn = 16 << i;
        constexpr double kStart[4] = {1.2, 1.5, 0.7, 6.3}, kBlock[4] = {0.225, 0.242, 0.272, 0.293}, kEnd[4] = {1.2, 1.5, 3.1, 0.0};
        if (bn > 16 && bn / 2 >= p.T && !(p.x[0].transposed && bn <= 64)) break;  // the width below holds all tokens
        if (p.x[0].transposed && bn < 64) continue;  // (a box of transposed X is 64 tokens)
        const int64_t tiles = ceil_div(p.R, gated ? 64 : kTile) * ceil_div(p.T, bn) * (two ? 2 : 1), slots = 2 * sm_count;
        for (int splits : {1, 2, 3, 4, 6, 8}) {
            if (splits * (keep8 ? 2 : 1) > kMaxSplits) break;  // (two tiles a cluster)
            if (splits > 1 && (splits > num_kb || tiles * splits > slots)) break;
            const int64_t blocks = ceil_div(num_kb, splits), full = tiles * splits / slots, rest = tiles * splits % slots;
            auto wave = [&](int64_t active) {
                return static_cast<double>(blocks) * std::max(kBlock[i] + (active > sm_count ? 0.49 * bn / 128 : 0.0),
                                                              static_cast<double>(active * (kOperandBytes + bn * 128)) / 10.8e6) +
                       kEnd[i] + (keep8 ? 0.02 * bn : 0.0);
            };
            const double t = static_cast<double>(full) * wave(slots) + (rest > 0 ? wave(rest) : 0.0);
            consider({bn, splits, 0}, kStart[i] + std::max(t, memory) + (keep8 ? 1.8 : 0.0) +
                                          (splits > 1 ? 1.1 + (splits > 4 ? 0.7 : 0.0) + 0.0024 * bn * (splits - 1) : 0.0));
        }
    }
    return best;
}

// Up to 8 tokens; up to kFewTokens where one round of its CTAs, two an SM, holds all rows, and, of a gated pair, where K is
// short. 12 tokens, few-token kernel and narrow tiles (us): 1024 x 1024 2.5 and 5.2, 2200 x 11008 11.8 and 14.0, 4500 x 11008
// 20.9 and 22.5, 6000 x 5000 18.4 and 16.0; gated 1024 x 1024 3.4 and 6.0, 1024 x 2500 7.6 and 8.8, 1024 x 11008 17.1 and 14.4,
// 3000 x 250 4.8 and 3.7. 8 tokens: 0.4 to 0.95 of the narrow tiles' time everywhere (64 .. 9000 rows, K = 250 .. 11008).
bool few_tokens(const ProductArgs& p, int sm_count) {
    const bool gated = p.kind == kGatedPair;
    if ((p.kind != kOneProduct && !gated) || p.keep == kKeep8 || p.x[0].transposed || p.w[0].transposed) return false;
    return p.T <= 8 || (p.T <= kFewTokens && p.R <= static_cast<int64_t>(gated ? 16 : 32) * sm_count && (!gated || p.K <= 2560));
}

}  // namespace

TilePlan plan_product(const ProductArgs& p, int sm_count) {
    return few_tokens(p, sm_count) && p.skip_stage < 0 ? TilePlan{kFewPlan, 1, 0} : plan_tiles(p, sm_count);
}

cudaError_t take_product_status(int* code, cudaStream_t stream) {
    int words[3] = {0, 0, 0};
    cudaError_t e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(words, g_status, sizeof(words));
    *code = words[kStatusCode];
    if (e == cudaSuccess && *code != 0) {
        const int clear[3] = {0, 0, 0};
        e = cudaMemcpyToSymbol(g_status, clear, sizeof(clear));
    }
    return e;
}

cudaError_t launch_product(const ProductArgs& p, const TilePlan& plan, int sm_count, cudaStream_t stream) {
    if (p.K > 0 && plan.bn == kFewPlan) return launch_few_tokens(p, sm_count, stream);
    GemmArgs a{};
    OutArgs& o = a.o;
    auto rows_aligned = [](const void* q, int64_t ld_bytes, int n) {
        return q == nullptr || (reinterpret_cast<uintptr_t>(q) % n == 0 && ld_bytes % n == 0);
    };
    const int e = p.y_type == VNM_F32 ? 4 : 2, k = p.keep == kKeep8 ? 1 : 2;
    o.T = p.T;
    o.R = p.R;
    o.y_vec = o.res_vec = true;
    for (int i = 0; i < (p.kind == kTwoByRows ? 2 : 1); ++i) {
        o.y[i] = p.y[i];
        o.res[i] = p.residual[i];
        o.y_vec = o.y_vec && rows_aligned(p.y[i], p.ld_y * e, 16);
        o.res_vec = o.res_vec && rows_aligned(p.residual[i], p.ld_residual * e, 16);
    }
    o.y_tma = o.y_vec;
    auto keep_aligned = [&](int n) {
        return p.keep == kKeepNone || (rows_aligned(p.g.p, p.g.ld * k, n) && rows_aligned(p.u.p, p.u.ld * k, n));
    };
    o.keep_vec = keep_aligned(8 * k);
    o.keep_tma = p.keep != kKeepNone && keep_aligned(16);
    o.bias = p.bias;
    o.ld_y = p.ld_y;
    o.ld_res = p.ld_residual;
    o.y_type = p.y_type;
    o.bias_type = p.bias_type;
    o.act = p.act;
    o.keep = p.keep;
    o.e5m2 = p.e5m2;
    o.g = p.g;
    o.u = p.u;
    if (p.K == 0) {
        const int64_t n = std::min<int64_t>(ceil_div(p.T * ceil_div(p.R, 8), 256), 16 * sm_count);
        return launch_early(dense_empty_kernel, n, 256, 0, 1, stream, o, static_cast<int>(p.kind));
    }
    a.kind = p.kind;
    a.num_kb = static_cast<int>(ceil_div(p.K, kBlockK));
    a.total_kb = a.num_kb * (p.kind == kSumOfTwo ? 2 : 1);
    a.chunk_kb = std::min(a.total_kb, p.y_type == VNM_F32 || p.keep == kKeep8 ? kChunk : kLongChunk);
    a.x_t = p.x[0].transposed;
    a.w_t = p.w[0].transposed;
    a.beside = p.beside;
    a.next_beside = p.next_beside;
    a.status = p.status;
    a.skip_stage = p.skip_stage;
    const bool gated = p.kind == kGatedPair;
    if (plan.bn == 0 && plan.splits > 1)
        return gated ? run_pair<true, true, true, false>(p, a, plan.tile_n, plan.splits, sm_count, stream)
                     : run_pair<false, true, true, false>(p, a, plan.tile_n, plan.splits, sm_count, stream);
    if (plan.bn == 0) {
        const bool aligned = o.y_tma && o.res_vec && p.R * e % 16 == 0 && (p.keep == kKeepNone || (o.keep_tma && p.R * k % 16 == 0));
        const bool sum = a.chunk_kb < a.total_kb || p.keep == kKeep8;
        return gated ? run_pair<true>(p, a, sum, aligned, plan.tile_n, sm_count, stream)
                     : run_pair<false>(p, a, sum, aligned, plan.tile_n, sm_count, stream);
    }
    return gated ? run_narrow<true>(plan.bn, p, a, plan.splits, stream) : run_narrow<false>(plan.bn, p, a, plan.splits, stream);
}

}  // namespace vnm
