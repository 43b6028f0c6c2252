// Dense Linear layer on block-scaled 8-bit operands:
//
//   Y[t][r] = act(sum_b xs[t, b] ws[r', b] (sum_{k in b} xq[t][k] wq[r][k]) + bias[r])
//
// The inner sums are 8-bit tensor-core products of one K block of 128
// (tcgen05.mma kind::f8f6f4, 4 MMAs of K = 32) into a TMEM buffer of their own;
// the outer sum is formed in registers, where each element of the buffer is
// scaled as it is added in fp32. So the MMAs of block b + 1 run while block b
// is added up, and no scale ever has to be a power of two.
//
// The kernel sees P (128 rows a CTA, the MMA's M side) times Q (BN rows a tile,
// the N side): P = X, Q = W for many tokens, P = W, Q = X for few of them, where
// the weights' rows then fill the tensor cores' rows and BN fits the tokens.
// Few tiles split K over the CTAs of a cluster, which add their sums up through
// distributed shared memory in rank order. Many tiles are taken by pairs of CTAs
// (cta_group::2): 256 x 256 outputs a pair, each CTA loading its own 128 rows of
// P and half of Q, so that a K block costs an SM 32 KB of loads instead of 48.
//
//   warp 0     TMA producer: a stage is 128 rows of P and the CTA's rows of Q by
//              128 bytes of K, 128B swizzle.
//   warp 1     TMEM owner and MMA issuer (one thread; of a pair, the first CTA's).
//   warps 2, 3 the K blocks' scales of Q into a shared-memory ring, where the tile has
//              more than one or two of them (any strides; four blocks at once where
//              they are 16 aligned bytes).
//   warps 4..  add up: thread = row of P, whose scale it loads two blocks ahead; 4
//              warps, or 8 with half the columns each.
// Every mbarrier wait is bounded.
//
// Measured: 8192 tokens, 11008 x 4096, bf16 out: 287-302 us, 2.45-2.57 PFLOP/s, 1.3-1.4 of
// the dense bf16 product's rate. The loads and MMAs alone run in 196 us, the sums alone
// (TMEM loads, 32768 fp32 FMAs a K block and SM, barriers) in 250: with two TMEM buffers
// a K block's MMAs wait for the sums of the block before last (at 4096 x 4096 x 4096 the
// tensor pipe is busy for 53 % of the SMs' active cycles). Bias and
// GELU add 105 us.
// Scales on both sides (4096 x 1024 outputs over 8192 tokens, fp32): 47.7 us. 16 tokens,
// 11008 x 4096: 13.7 us, 3.3 TB/s, a chain of 16 K blocks a CTA and 5 us of start and end.
#include <algorithm>
#include <atomic>

#include "vnm_dense.h"
#include "vnm_fp8.cuh"
#include "vnm_internal.h"
#include "vnm_ptx.cuh"
#include "vnm_umma.cuh"

namespace vnm {
namespace {

constexpr int kTileM = 128;
constexpr int kMaxSplits = 8;
constexpr int kHelpers = 4;  // warps before the adding ones
constexpr int kMaxDevicesFl = 64;
constexpr int kStoreBox = 32 * 128;  // bytes of a TMA store: 32 rows x 128 bytes

// BN: columns of the tile; ONE: every thread's columns lie in one 128-row block
// of Q, with one scale; CG: CTAs of a tile (1, or 2 for a pair).
template <int BN, bool ONE, int CG>
struct FlCfg {
    static constexpr int kPBytes = kTileM * 128;
    static constexpr int kQRows = BN / CG;
    static constexpr int kQBytes = kQRows * 128;
    static constexpr int kStageBytes = kPBytes + kQBytes;
    // narrow tiles: two CTAs an SM, whose waits overlap
    static constexpr int kCtas = BN <= 64 ? 2 : 1;
    static constexpr int kStages = CG == 2 ? 4 : BN == 128 ? 6 : BN == 64 ? 4 : BN == 32 ? 5 : 6;
    static constexpr int kAcc = BN == 256 ? 2 : 4;  // TMEM buffers
    static constexpr int kTmemCols = kAcc * BN;
    static constexpr int kAddWarps = BN >= 128 ? 8 : 4;
    static constexpr int kCols = BN * 4 / kAddWarps;  // columns a thread adds up
    static constexpr int kLoad = BN >= 128 ? 32 : 16;  // columns of one TMEM load
    static constexpr int kThreads = 32 * (kHelpers + kAddWarps);
    // Registers: 128 sums and two loads of 32 columns do not fit the 168 that 12
    // warps get; the adding warps take what the helper warps leave. The shares
    // add up to the launch's (in warps: 4 x 56 + 8 x 224 = 4 x 104 + 8 x 200 = 12 x 168).
    static constexpr bool kSplitRegs = kCols == 128;
    static constexpr int kLaunchRegs = 168, kHelperRegs = ONE ? 56 : 104, kAddRegs = ONE ? 224 : 200;
    static_assert(!kSplitRegs || kHelpers * kHelperRegs + kAddWarps * kAddRegs == (kHelpers + kAddWarps) * kLaunchRegs,
                  "register shares");
    // FRAG: a pair whose columns have a scale each. A thread then holds 4 rows x 32
    // columns (two neighbours of every 8) instead of a row x 128, and reads 32 of Q's
    // scales a K block instead of 128: as one row a thread, their broadcasts from
    // shared memory took 1 us a K block.
    static constexpr bool kFrag = CG == 2 && !ONE;
    // Q's scales (ONE reads its one scale itself), FRAG: and P's; they take about as long to arrive
    // as an operand stage
    static constexpr int kScaleSlots = ONE ? 0 : 8;
    static constexpr int kScaleFloats = BN + (kFrag ? kTileM : 0);
    // a pair's outputs leave by TMA stores, from two boxes of 32 rows x 128 bytes for each adding warp
    static constexpr int kStoreBytes = CG == 2 ? kAddWarps * 2 * kStoreBox : 0;
    // no CTA waits for TMEM that another of this kernel holds: either the CTAs that
    // share an SM leave each other room, or the shared memory keeps a second one out
    static constexpr int kSmem = kStages * kStageBytes + kStoreBytes + kScaleSlots * kScaleFloats * 4 + 1024;
    static_assert(kCtas * kTmemCols <= 512, "TMEM of the CTAs that share an SM");
    static_assert(kCtas == 2 ? 2 * (kSmem + 2048) <= 228 * 1024 : kSmem > 116 * 1024 && kSmem <= 226 * 1024, "shared memory");
    static_assert(CG == 2 || kTileM * BN * 4 <= kStages * kStageBytes, "the split's sums fit the stage ring");
};

struct FlArgs {
    int64_t m, n;
    int num_kb, splits, kb_per_split;
    int m_tiles, n_tiles, tiles;
    uint32_t idesc;
    ScaleView ps, qs;
    bool quad_scales;  // four blocks' scales of a row are 16 aligned bytes
    void* y;
    int64_t y_ms, y_ns;
    int y_type;
    bool y_tma;    // Y's rows start on 16 bytes: pairs write it by TMA stores,
    bool y_ends;   // and end on 16: the last columns too
    const void* bias;
    int bias_type;
    bool bias_on_m;
    int act;
    int* status;
    int skip_stage;  // tests of the bounded waits only (-1: none)
};

// Instruction descriptor of kind::f8f6f4 with an fp32 accumulator, both
// operands K-major: bits 4-5 D format (1 = f32), 7-9 / 10-12 A / B format
// (0 = e4m3, 1 = e5m2), 17-22 N >> 3, 24-28 M >> 4.
constexpr uint32_t fp8_idesc(int m, int n, bool a_e5m2, bool b_e5m2) {
    return (1u << 4) | ((a_e5m2 ? 1u : 0u) << 7) | ((b_e5m2 ? 1u : 0u) << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

// D[tmem] (+)= A[smem] x B[smem], 8-bit inputs, fp32 D; CG = 2: of a pair, each
// CTA holding half the rows of A, of B and of D at the same addresses.
template <int CG>
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    if (CG == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// 4-byte asynchronous copy global -> shared (0 where !valid).
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, bool valid) {
    const uint32_t n = valid ? 4u : 0u;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// Output (m, n) from its sum.
__device__ __forceinline__ void store_one(const FlArgs& a, int64_t m, int64_t n, float v) {
    if (a.bias) v += load_any(a.bias, a.bias_type, a.bias_on_m ? m : n);
    store_any(a.y, a.y_type, m * a.y_ms + n * a.y_ns, activate(a.act, v));
}

// One copy of this code: unrolled over a thread's columns, GELU's alone is tens of
// KB, and fetching it took 20 us a tile.
__device__ __noinline__ void gelu16(float (&v)[16]) {
#pragma unroll
    for (int u = 0; u < 16; ++u) v[u] = activate(VNM_ACT_GELU, v[u]);
}

// 16 outputs of row m from their finished sums (narrow tiles: neighbouring lanes' rows are
// neighbours in Y).
__device__ __noinline__ void store_any16(const FlArgs& a, int64_t m, int64_t n, float (&v)[16]) {
#pragma unroll
    for (int u = 0; u < 16; ++u)
        if (n + u < a.n) store_any(a.y, a.y_type, m * a.y_ms + (n + u) * a.y_ns, v[u]);
}

// The bias of columns n, n + 1 (the last one's past the edge).
__device__ __noinline__ float2 bias2(const FlArgs& a, int64_t n) {
    return make_float2(load_any(a.bias, a.bias_type, min(n, a.n - 1)), load_any(a.bias, a.bias_type, min(n + 1, a.n - 1)));
}

// A staged box (32 rows x 128 bytes, 128B-swizzled) to Y's rows m0 .. and columns
// n0 .., by a warp, 4 bytes a lane: whole words where the row's address allows them.
template <bool F32>
__device__ __noinline__ void copy_box(const FlArgs& a, uint32_t buf, int m0, int n0, int lane) {
    const int rows = static_cast<int>(min(static_cast<int64_t>(32), a.m - m0));
    const int64_t n = n0 + (F32 ? lane : 2 * lane);
#pragma unroll 4
    for (int r = 0; r < rows; ++r) {
        uint32_t v;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(buf + 128 * r + 16 * ((lane >> 2) ^ (r & 7)) + 4 * (lane & 3)));
        const int64_t at = static_cast<int64_t>(m0 + r) * a.y_ms + n;
        if (F32) {
            if (n < a.n) static_cast<uint32_t*>(a.y)[at] = v;
        } else {
            uint16_t* p = static_cast<uint16_t*>(a.y) + at;
            if (n + 1 < a.n && (reinterpret_cast<uintptr_t>(p) & 3) == 0) {
                *reinterpret_cast<uint32_t*>(p) = v;
            } else {
                if (n < a.n) p[0] = static_cast<uint16_t>(v);
                if (n + 1 < a.n) p[1] = static_cast<uint16_t>(v >> 16);
            }
        }
    }
}

__device__ __forceinline__ void st_shared_v2(uint32_t addr, float x, float y) {
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Tiles in groups of kGroupM row tiles, row tiles fastest: the CTAs that run
// together share a few tiles of both operands in L2.
constexpr int kGroupM = 8;
__device__ __forceinline__ void tile_at(const FlArgs& a, int tile, int& mt, int& nt) {
    const int per_group = kGroupM * a.n_tiles;
    const int g = tile / per_group, r = tile - g * per_group;
    const int rows = min(kGroupM, a.m_tiles - g * kGroupM);
    nt = r / rows;
    mt = g * kGroupM + (r - nt * rows);
}

// Status words of the calls that were given none (of the device's all).
__device__ int g_status[3];

// F32: Y is fp32 (for a pair's staged output).
template <int BN, bool ONE, int CG, bool F32>
__global__ void __launch_bounds__(FlCfg<BN, ONE, CG>::kThreads, FlCfg<BN, ONE, CG>::kCtas)
    fp8_linear_kernel(const __grid_constant__ CUtensorMap tm_p, const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ FlArgs a) {
    using Cfg = FlCfg<BN, ONE, CG>;
    constexpr int ST = Cfg::kStages, ACC = Cfg::kAcc, SS = Cfg::kScaleSlots, COLS = Cfg::kCols, LD = Cfg::kLoad;
    constexpr int SSB = SS > 0 ? SS : 1;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[ST];   // the stage's operands have landed (a pair's: in the first CTA)
    // the MMAs of the stage are done: its TMEM buffer is full and its operands are free
    __shared__ __align__(8) uint64_t done_bar[ST];
    __shared__ __align__(8) uint64_t acce_bar[ACC];  // the TMEM buffer has been read (a pair's: in the first CTA)
    __shared__ __align__(8) uint64_t scf_bar[SSB], sce_bar[SSB];  // Q's scales have landed, have been read
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* const smem_gen = smem_raw + (smem_base - smem_u32(smem_raw));
    float* const scales = reinterpret_cast<float*>(smem_gen + ST * Cfg::kStageBytes + Cfg::kStoreBytes);  // [SS][kScaleFloats]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pair_rank = CG == 2 ? static_cast<int>(blockIdx.x & 1) : 0;
    // this CTA's tiles and K blocks: every role walks the same sequence
    const int rank = CG == 1 && a.splits > 1 ? static_cast<int>(blockIdx.x) % a.splits : 0;
    const int tile0 = static_cast<int>(blockIdx.x) / (CG == 2 ? 2 : a.splits);
    const int tile_step = a.splits > 1 ? a.tiles : static_cast<int>(gridDim.x) / CG;
    const int kb0 = rank * a.kb_per_split;
    const int kb1 = min(a.num_kb, kb0 + a.kb_per_split);

    const int early = CG == 1 ? min(ST, kb1 - kb0) : 0;  // stages loaded before the setup is over

    // one stage's loads into its slot (a single CTA's)
    auto load_stage = [&](int slot, int kb, int prow, int qrow) {
        const uint32_t fb = smem_u32(&full_bar[slot]), sp = smem_base + slot * Cfg::kStageBytes;
        mbar_arrive_expect_tx(fb, Cfg::kStageBytes);
        tma_load_2d(sp, &tm_p, kb * 128, prow, fb);
        tma_load_2d(sp + Cfg::kPBytes, &tm_q, kb * 128, qrow, fb);
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(smem_u32(&full_bar[s]), 1);
            mbar_init(smem_u32(&done_bar[s]), 1);
        }
        for (int s = 0; s < ACC; ++s) mbar_init(smem_u32(&acce_bar[s]), CG * Cfg::kAddWarps);
        for (int s = 0; s < SS; ++s) {
            mbar_init(smem_u32(&scf_bar[s]), 64);
            mbar_init(smem_u32(&sce_bar[s]), Cfg::kAddWarps);
        }
        abort_flag = 0;
        fence_barrier_init();
        // the first stages need no other thread: their latency covers the TMEM allocation
        int mt, nt;
        tile_at(a, tile0, mt, nt);
        for (int k = 0; k < early; ++k)
            if (k != a.skip_stage || blockIdx.x != 0) load_stage(k, kb0 + k, mt * kTileM, nt * BN);
    }
    if (warp == 1) tmem_alloc_group<CG>(smem_u32(&tmem_slot), Cfg::kTmemCols);
    tc_fence_before_sync();
    __syncthreads();
    if (CG == 2) cluster_sync_all();  // both CTAs' barriers and TMEM exist
    tc_fence_after_sync();
    const uint32_t tmem = tmem_slot;
    volatile int* abort = &abort_flag;

    if (Cfg::kSplitRegs && warp < kHelpers) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kHelperRegs));
    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        int it = 0, slot = 0;
        uint32_t phase = 1;
        bool run = true;
        for (int tile = tile0; tile < a.tiles && run; tile += tile_step) {
            int mt, nt;
            tile_at(a, tile, mt, nt);
            const int prow = (mt * CG + pair_rank) * kTileM, qrow = nt * BN + pair_rank * Cfg::kQRows;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                if (it >= early && !mbar_wait_warp(smem_u32(&done_bar[slot]), phase, abort)) {
                    run = false;
                    break;
                }
                if (it >= early && elect_one() && (it != a.skip_stage || blockIdx.x != 0)) {
                    if (CG == 2) {
                        const uint32_t fb = smem_u32(&full_bar[slot]);
                        const uint32_t sp = smem_base + slot * Cfg::kStageBytes;
                        // the second CTA's bytes may arrive before the first CTA expects them: the
                        // phase cannot end before that CTA's own arrival
                        const uint32_t lead = dsmem_map(fb, 0);
                        if (pair_rank == 0) mbar_arrive_expect_tx(fb, 2 * Cfg::kStageBytes);
                        tma_load_2d_pair(sp, &tm_p, kb * 128, prow, lead);
                        tma_load_2d_pair(sp + Cfg::kPBytes, &tm_q, kb * 128, qrow, lead);
                    } else {
                        load_stage(slot, kb, prow, qrow);
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
            if (pair_rank == 0) {
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
        // both operands K-major, 128B swizzle, 128-byte rows, 8-row groups 1024 bytes
        // apart; MMA k-step s (K = 32) takes bytes 32s .. 32s + 31 of every row
        const uint64_t pdesc = make_smem_desc(smem_base, 16, 1024, kLayoutSw128);
        const uint64_t qdesc = make_smem_desc(smem_base + Cfg::kPBytes, 16, 1024, kLayoutSw128);
        int it = 0, slot = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 1;
        bool run = pair_rank == 0;
        for (int tile = tile0; tile < a.tiles && run; tile += tile_step) {
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait2(smem_u32(&full_bar[slot]), phase, smem_u32(&acce_bar[acc]),
                                                        acc_phase, abort))) {
                    run = false;
                    break;
                }
                tc_fence_after_sync();
                if (elect_one()) {
                    const uint64_t off = static_cast<uint64_t>((slot * Cfg::kStageBytes) >> 4);
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        tc_mma_f8<CG>(tmem + acc * BN, pdesc + off + 2 * s, qdesc + off + 2 * s, a.idesc,
                                      s > 0 ? 1u : 0u);
                    tc_commit_group<CG>(smem_u32(&done_bar[slot]));
                }
                __syncwarp();
                if (++slot == ST) {
                    slot = 0;
                    phase ^= 1;
                }
                if (++acc == ACC) {
                    acc = 0;
                    acc_phase ^= 1;
                }
            }
        }
        // every MMA issued is done before TMEM goes back
        if (it > 0) mbar_drain(smem_u32(&done_bar[(it - 1) % ST]), static_cast<uint32_t>((it - 1) / ST) & 1u);
    } else if (warp < kHelpers && !ONE) {
        // ------------------------------------------------ scales, by warps 2 and 3
        constexpr int F = Cfg::kScaleFloats, kPer = (F + 63) / 64;  // scales of a slot, and a lane's share
        const int first = 32 * (warp - 2) + lane;                   // the lane's: first, first + 64, ...
        int it = 0;
        bool run = true;
        for (int tile = tile0; tile < a.tiles && run; tile += tile_step) {
            int mt, nt;
            tile_at(a, tile, mt, nt);
            const int64_t n0 = static_cast<int64_t>(nt) * BN, m0 = static_cast<int64_t>(mt * CG + pair_rank) * kTileM;
            // scale i of a slot at block 0; null past the operand's edge
            auto place = [&](int i) -> const float* {
                const bool q = i < BN;
                const int64_t r = q ? n0 + i : m0 + (i - BN);
                if (i >= F || r >= (q ? a.n : a.m)) return nullptr;
                return q ? a.qs.p + (r >> a.qs.shift) * a.qs.rs : a.ps.p + (r >> a.ps.shift) * a.ps.rs;
            };
            for (int kb = kb0; kb < kb1 && run;) {
                // four blocks of a row in one load where the scales' layout allows it: one by one,
                // a weight gradient's 384 scales a block cost a third of its time
                const int many = a.quad_scales && (kb & 3) == 0 && kb + 4 <= kb1 ? 4 : 1;
                for (int u = 0; u < many && run; ++u)
                    run = mbar_wait_warp(smem_u32(&sce_bar[(it + u) % SSB]), (static_cast<uint32_t>((it + u) / SSB) & 1u) ^ 1u,
                                         abort);
                if (!run) break;
                if (many == 4) {
                    float4 v[kPer];
#pragma unroll
                    for (int j = 0; j < kPer; ++j) {
                        const float* p = place(first + 64 * j);
                        v[j] = p ? *reinterpret_cast<const float4*>(p + kb) : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        float* dst = scales + (it + u) % SSB * F;
#pragma unroll
                        for (int j = 0; j < kPer; ++j)
                            if (first + 64 * j < F)
                                dst[first + 64 * j] = u == 0 ? v[j].x : u == 1 ? v[j].y : u == 2 ? v[j].z : v[j].w;
                        mbar_arrive(smem_u32(&scf_bar[(it + u) % SSB]));
                    }
                } else {
                    const uint32_t dst = smem_u32(scales + it % SSB * F);
#pragma unroll
                    for (int j = 0; j < kPer; ++j) {
                        const int i = first + 64 * j;
                        const float* p = place(i);
                        if (i < F) cp_async_4(dst + 4 * i, p ? p + kb * (i < BN ? a.qs.cs : a.ps.cs) : a.qs.p, p != nullptr);
                    }
                    cp_async_arrive_noinc(smem_u32(&scf_bar[it % SSB]));
                }
                kb += many;
                it += many;
            }
        }
        cp_async_wait_all();
    } else if (warp >= kHelpers) {
        // ------------------------------------------------ adding up
        if (Cfg::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kAddRegs));
        const int quarter = warp & 3;                   // TMEM lanes 32 quarter ..
        const int row = 32 * quarter + lane;            // row of the tile
        const int col0 = ((warp - kHelpers) >> 2) * COLS;  // first column of the tile
        const uint32_t lane_addr = static_cast<uint32_t>(32 * quarter) << 16;
        const uint32_t acce_lead = CG == 2 ? dsmem_map(smem_u32(&acce_bar[0]), 0) : 0;
        // The scales of this thread's row and, of a ONE tile, of its columns are loaded two
        // K blocks ahead, over the end of the tile as well. Rows and columns past the
        // edges take the last one's: their sums are not stored.
        const float *cur_p = a.ps.p, *cur_q = a.qs.p, *next_p = a.ps.p, *next_q = a.qs.p;
        int m0 = 0, n0 = 0, next_m0 = 0, next_n0 = 0;  // the warp's first row, the thread's first column
        auto point = [&](int tile) {
            int mt, nt;
            tile_at(a, tile, mt, nt);
            next_m0 = (mt * CG + pair_rank) * kTileM + 32 * quarter;
            next_n0 = nt * BN + col0;
            next_p = a.ps.p + (min(static_cast<int64_t>(next_m0) + lane, a.m - 1) >> a.ps.shift) * a.ps.rs + kb0 * a.ps.cs;
            if (ONE) next_q = a.qs.p + (min(static_cast<int64_t>(next_n0), a.n - 1) >> a.qs.shift) * a.qs.rs + kb0 * a.qs.cs;
        };
        float p1 = 0.f, p2 = 0.f, q1 = 0.f, q2 = 0.f;  // of the next K block and the one after it
        point(tile0);
        cur_p = next_p;
        cur_q = next_q;
        const bool two = kb1 - kb0 >= 2;
        if (!Cfg::kFrag && kb0 < kb1) {
            p1 = *cur_p;
            if (ONE) q1 = *cur_q;
        }
        if (!Cfg::kFrag && two) {
            p2 = *(cur_p += a.ps.cs);
            if (ONE) q2 = *(cur_q += a.qs.cs);
        }
        int it = 0, stage = 0;
        uint32_t phase = 0;
        bool run = true;
        for (int tile = tile0; tile < a.tiles && run; tile += tile_step) {
            m0 = next_m0;
            n0 = next_n0;
            if (tile + tile_step < a.tiles) point(tile + tile_step);
            float sum[COLS];
#pragma unroll
            for (int c = 0; c < COLS; ++c) sum[c] = 0.f;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int acc = it % ACC, slot = it % SSB;
                const float sp = p1, sq1 = q1;
                if (!Cfg::kFrag) {
                    p1 = p2;
                    q1 = q2;
                    if (kb + 2 == kb1 || !two) {
                        cur_p = next_p;
                        cur_q = next_q;
                    } else {
                        cur_p += a.ps.cs;
                        cur_q += a.qs.cs;
                    }
                    p2 = *cur_p;
                    if (ONE) q2 = *cur_q;
                    if (!two) {  // one block a tile: the next tile's is the next one
                        p1 = p2;
                        q1 = q2;
                    }
                }
                const uint32_t done = smem_u32(&done_bar[stage]);
                const bool ok = ONE ? mbar_wait(done, phase, abort)
                                    : mbar_wait2(smem_u32(&scf_bar[slot]), static_cast<uint32_t>(it / SSB) & 1u, done,
                                                 phase, abort);
                if (++stage == ST) {
                    stage = 0;
                    phase ^= 1;
                }
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    run = false;
                    break;
                }
                tc_fence_after_sync();
                const float* sq = scales + slot * Cfg::kScaleFloats + col0;
                const float s1 = ONE ? sp * sq1 : sp;
                const uint32_t taddr = tmem + lane_addr + acc * BN + col0;
                // all read: the MMAs may have the buffer back
                auto release = [&] {
                    tc_fence_before_sync();
                    __syncwarp();
                    if (elect_one()) {
                        if (CG == 2)
                            mbar_arrive_cluster(acce_lead + 8 * acc);
                        else
                            mbar_arrive(smem_u32(&acce_bar[acc]));
                    }
                };
                // the next columns are on their way while these are added
                if constexpr (Cfg::kFrag) {
                    // chunk x: rows 16 (x & 1) of the warp's 32, columns 32 (x / 2)
                    const float *fp = scales + slot * Cfg::kScaleFloats + BN + 32 * quarter + (lane >> 2),
                                *fq = sq + 2 * (lane & 3);
                    const float rows[4] = {fp[0], fp[8], fp[16], fp[24]};
                    auto at = [&](int x) { return taddr + (static_cast<uint32_t>(16 * (x & 1)) << 16) + 32 * (x / 2); };
                    uint32_t v[2][16];
                    tmem_ld_frag(at(0), v[0]);
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        uint32_t(&cur)[16] = v[x & 1];
                        tmem_wait_ld(cur);
                        if (x + 1 < 8)
                            tmem_ld_frag(at(x + 1), v[(x + 1) & 1]);
                        else
                            release();
                        const float top = rows[2 * (x & 1)], low = rows[2 * (x & 1) + 1];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 q = *reinterpret_cast<const float2*>(fq + 32 * (x / 2) + 8 * j);
                            float* d = sum + 16 * x + 4 * j;
                            d[0] = fmaf(__uint_as_float(cur[4 * j]), top * q.x, d[0]);
                            d[1] = fmaf(__uint_as_float(cur[4 * j + 1]), top * q.y, d[1]);
                            d[2] = fmaf(__uint_as_float(cur[4 * j + 2]), low * q.x, d[2]);
                            d[3] = fmaf(__uint_as_float(cur[4 * j + 3]), low * q.y, d[3]);
                        }
                    }
                } else {
                    uint32_t v[2][LD];
                    tmem_ld(taddr, v[0]);
#pragma unroll
                    for (int c = 0; c < COLS; c += LD) {
                        uint32_t(&cur)[LD] = v[(c / LD) & 1];
                        tmem_wait_ld(cur);
                        if (c + LD < COLS)
                            tmem_ld(taddr + c + LD, v[(c / LD + 1) & 1]);
                        else
                            release();
#pragma unroll
                        for (int u = 0; u < LD; u += 4) {
                            float4 q4 = make_float4(1.f, 1.f, 1.f, 1.f);
                            if (!ONE) q4 = *reinterpret_cast<const float4*>(sq + c + u);
                            sum[c + u] = fmaf(__uint_as_float(cur[u]), ONE ? s1 : s1 * q4.x, sum[c + u]);
                            sum[c + u + 1] = fmaf(__uint_as_float(cur[u + 1]), ONE ? s1 : s1 * q4.y, sum[c + u + 1]);
                            sum[c + u + 2] = fmaf(__uint_as_float(cur[u + 2]), ONE ? s1 : s1 * q4.z, sum[c + u + 2]);
                            sum[c + u + 3] = fmaf(__uint_as_float(cur[u + 3]), ONE ? s1 : s1 * q4.w, sum[c + u + 3]);
                        }
                    }
                }
                if (!ONE) {
                    __syncwarp();
                    if (elect_one()) mbar_arrive(smem_u32(&sce_bar[slot]));
                }
            }
            if (!run) break;
            if (CG == 1 && a.splits > 1) {
                // the stage ring is free: this tile's MMAs are done with it
                float* part = reinterpret_cast<float*>(smem_gen);
#pragma unroll
                for (int c = 0; c < COLS; ++c) part[(col0 + c) * kTileM + row] = sum[c];
                continue;
            }
            const int64_t m = static_cast<int64_t>(m0) + lane;
            if (Cfg::kFrag && a.bias) {
#pragma unroll
                for (int x = 0; x < COLS / 16; x += 2) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 b = bias2(a, static_cast<int64_t>(n0) + 16 * x + 8 * j + 2 * (lane & 3));
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            sum[16 * x + 16 * (h / 2) + 4 * j + 2 * (h & 1)] += b.x;
                            sum[16 * x + 16 * (h / 2) + 4 * j + 2 * (h & 1) + 1] += b.y;
                        }
                    }
                }
            } else if (a.bias) {
                // the bias of the row, or of columns lane, lane + 32, ... (the sum over a
                // cluster adds it by itself)
                float bias[(COLS + 31) / 32];
#pragma unroll
                for (int i = 0; i < (COLS + 31) / 32; ++i) {
                    const int64_t n = min(static_cast<int64_t>(n0) + 32 * i + lane, a.n - 1);
                    bias[i] = load_any(a.bias, a.bias_type, a.bias_on_m ? min(m, a.m - 1) : n);
                }
#pragma unroll
                for (int c = 0; c < COLS; ++c)
                    sum[c] += a.bias_on_m ? bias[0] : __shfl_sync(0xFFFFFFFFu, bias[c / 32], c & 31);
            }
            if (a.act == VNM_ACT_RELU) {
#pragma unroll
                for (int c = 0; c < COLS; ++c) sum[c] = activate(VNM_ACT_RELU, sum[c]);
            } else if (a.act == VNM_ACT_GELU && (Cfg::kFrag || m < a.m)) {
#pragma unroll
                for (int c = 0; c < COLS; c += 16) {
                    float v[16];
#pragma unroll
                    for (int u = 0; u < 16; ++u) v[u] = sum[c + u];
                    gelu16(v);
#pragma unroll
                    for (int u = 0; u < 16; ++u) sum[c + u] = v[u];
                }
            }
            if (CG == 2) {
                // 128 bytes of 32 rows at a time, 128B-swizzled, then one TMA store (which
                // leaves out what lies past Y's edges), or, where Y's rows do not start on 16 bytes and for
                // the last columns of rows that do not end on 16 (a TMA store that ends inside 16 bytes writes all
                // of them), a copy row by row. 8192 x 11007 over 4096 in rows of 11008: 288 us in bf16 and 307 in fp32, where
                // a copy of all boxes took 378 and 481; 2500 x 2001 over 256 12.5 and 11.8, 19.5 and 28.3.
                constexpr int kBoxCols = F32 ? 32 : 64;
                const bool bf16 = a.y_type == VNM_BF16;
                const uint32_t bufs = smem_base + ST * Cfg::kStageBytes + (warp - kHelpers) * 2 * kStoreBox;
                const uint32_t flip = lane & 7;
#pragma unroll
                for (int c = 0; c < COLS; c += kBoxCols) {
                    const uint32_t buf = bufs + (c / kBoxCols & 1) * kStoreBox, dst = buf + 128 * lane;
                    if (lane == 0) tma_store_wait_read();
                    __syncwarp();
                    if (Cfg::kFrag) {
                        const int g = lane >> 2, i = lane & 3;  // (rows g, g + 8, ...: all of the swizzle's row g)
#pragma unroll
                        for (int x = c / 16; x < (c + kBoxCols) / 16; ++x)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
#pragma unroll
                                for (int low = 0; low < 2; ++low) {
                                    const float *d = sum + 16 * x + 4 * j + 2 * low;
                                    const uint32_t to = buf + 128 * (16 * (x & 1) + g + 8 * low);
                                    const int col = 32 * (x / 2) + 8 * j - c;  // of the box
                                    if (F32)
                                        st_shared_v2(to + 16 * ((col / 4 + (i >> 1)) ^ g) + 8 * (i & 1), d[0], d[1]);
                                    else
                                        st_shared_u32(to + 16 * ((col / 8) ^ g) + 4 * i,
                                                      bf16 ? to_bf16x2(d[0], d[1]) : to_f16x2(d[0], d[1]));
                                }
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {  // 16 bytes each
                            uint32_t w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int e = c + j * kBoxCols / 8 + (F32 ? i : 2 * i);
                                w[i] = F32    ? __float_as_uint(sum[e])
                                       : bf16 ? to_bf16x2(sum[e], sum[e + 1])
                                              : to_f16x2(sum[e], sum[e + 1]);
                            }
                            st_shared_v4(dst + 16 * (j ^ flip), w[0], w[1], w[2], w[3]);
                        }
                    }
                    if (!a.y_tma || (!a.y_ends && n0 + c < a.n && n0 + c + kBoxCols > a.n)) {
                        __syncwarp();
                        copy_box<F32>(a, buf, m0, n0 + c, lane);
                        __syncwarp();
                        if (lane == 0) tma_store_commit();  // (an empty group: the waits count groups)
                        continue;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        // a box past Y's edges is an empty group: the waits count groups
                        if (m0 < a.m && n0 + c < a.n) tma_store_2d(&tm_y, n0 + c, m0, buf);
                        tma_store_commit();
                    }
                }
                continue;
            }
            if (m >= a.m) continue;
#pragma unroll
            for (int c = 0; c < COLS; c += 16) {
                float v[16];
#pragma unroll
                for (int u = 0; u < 16; ++u) v[u] = sum[c + u];
                store_any16(a, m, n0 + c, v);
            }
        }
        if (CG == 2 && lane == 0) tma_store_wait();
    }

    tc_fence_before_sync();
    __syncthreads();
    if (CG == 2) {
        cluster_sync_all();  // neither CTA leaves while the other's arrivals or MMAs may reach it
    } else if (a.splits > 1) {
        // add the cluster's sums, in rank order; each CTA takes its share of the columns
        cluster_sync_all();
        int mt, nt;
        tile_at(a, tile0, mt, nt);
        const int share = (BN + a.splits - 1) / a.splits, c0 = rank * share, c1 = min(BN, c0 + share);
        const int64_t n0 = static_cast<int64_t>(nt) * BN;
        // four rows of a column at a time
        for (int i = threadIdx.x; i < (c1 - c0) * (kTileM / 4); i += Cfg::kThreads) {
            const int c = c0 + i / (kTileM / 4), row = 4 * (i % (kTileM / 4));
            const int64_t m = static_cast<int64_t>(mt) * kTileM + row, n = n0 + c;
            if (m >= a.m || n >= a.n) continue;
            const uint32_t addr = smem_base + 4 * (c * kTileM + row);
            float4 v[kMaxSplits];
#pragma unroll
            for (int s = 0; s < kMaxSplits; ++s)
                if (s < a.splits) v[s] = dsmem_ld_v4(dsmem_map(addr, s));
            float4 sum = v[0];
#pragma unroll
            for (int s = 1; s < kMaxSplits; ++s)
                if (s < a.splits) {
                    sum.x += v[s].x;
                    sum.y += v[s].y;
                    sum.z += v[s].z;
                    sum.w += v[s].w;
                }
            float out[4] = {sum.x, sum.y, sum.z, sum.w};
            const int here = static_cast<int>(min(static_cast<int64_t>(4), a.m - m));
#pragma unroll 1
            for (int j = 0; j < here; ++j) store_one(a, m + j, n, out[j]);
        }
        cluster_sync_all();  // no CTA leaves while others read its sums
    }
    if (threadIdx.x == 0 && abort_flag) record_error(a.status ? a.status : g_status, VNM_ERR_TIMEOUT, 12);
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_group<CG>(tmem, Cfg::kTmemCols);
    }
}

// K = 0: act(bias).
__global__ void fp8_linear_empty_kernel(const FlArgs a) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < a.m * a.n;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x)
        store_one(a, i / a.n, i % a.n, 0.f);
}

// A row-major matrix as boxes of 128 bytes x `box_rows` rows, 128B swizzle; past
// its edges it reads as 0.
bool encode(CUtensorMap* tm, CUtensorMapDataType type, int elem, const void* base, int64_t cols, int64_t rows, int64_t ld,
            int box_rows) {
    return encode_2d(tm, type, base, cols, rows, ld * elem, 128 / elem, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int BN, bool ONE, int CG, bool F32 = false>
cudaError_t run(const Fp8LinearArgs& g, FlArgs a, int splits, int sm_count, cudaStream_t stream) {
    using Cfg = FlCfg<BN, ONE, CG>;
    a.m_tiles = static_cast<int>((g.m + CG * kTileM - 1) / (CG * kTileM));
    a.n_tiles = static_cast<int>((g.n + BN - 1) / BN);
    const int64_t tiles = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
    if (tiles * kMaxSplits > INT32_MAX) return cudaErrorInvalidValue;
    a.tiles = static_cast<int>(tiles);
    a.splits = splits;
    a.kb_per_split = (a.num_kb + splits - 1) / splits;
    a.idesc = fp8_idesc(CG * kTileM, BN, g.p_e5m2, g.q_e5m2);
    CUtensorMap tm_p, tm_q, tm_y;
    if (!encode(&tm_p, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.p, g.k, g.m, g.ld_p, kTileM) ||
        !encode(&tm_q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.q, g.k, g.n, g.ld_q, Cfg::kQRows))
        return cudaErrorInvalidValue;
    tm_y = tm_p;  // not used, unless:
    if (CG == 2 && a.y_tma) {
        const CUtensorMapDataType t = a.y_type == VNM_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                      : a.y_type == VNM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                            : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
        if (!encode(&tm_y, t, a.y_type == VNM_F32 ? 4 : 2, a.y, g.n, g.m, a.y_ms, 32)) return cudaErrorInvalidValue;
    }
    static std::atomic<bool> attr_set[kMaxDevicesFl];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevicesFl) return cudaErrorInvalidDevice;
    if (!attr_set[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(fp8_linear_kernel<BN, ONE, CG, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
        if (e != cudaSuccess) return e;
        if (Cfg::kSplitRegs) {
            // the shares are drawn from the launch's registers: never ask for more
            cudaFuncAttributes fa;
            if ((e = cudaFuncGetAttributes(&fa, fp8_linear_kernel<BN, ONE, CG, F32>)) != cudaSuccess) return e;
            if (fa.numRegs != Cfg::kLaunchRegs) return cudaErrorInvalidConfiguration;
        }
        attr_set[dev].store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    const int64_t ctas = splits > 1 ? tiles * splits : CG * std::min<int64_t>(tiles, std::max(1, sm_count * Cfg::kCtas / CG));
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(Cfg::kThreads);
    cfg.dynamicSmemBytes = Cfg::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(splits * CG);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = splits * CG > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fp8_linear_kernel<BN, ONE, CG, F32>, tm_p, tm_q, tm_y, a);
}

// How a product of T tokens and R outputs over num_kb K blocks is tiled: pairs
// of CTAs (bn = 0), X on the M side; or W on the M side, tiles of bn tokens, K over
// `splits` CTAs of a cluster.
struct TilePlan {
    int bn, splits;
};

// The times the plan compares, in us, fitted to measurements over T = 1 .. 8192,
// R = 300 .. 11008, K = 1024 .. 8192: a launch with its first loads and its last
// stores; then the longer of a CTA's chain of K blocks and of its tiles' loads from
// L2. At 4096 x 4096 (T, narrow, pairs): (64, 10.0, 20), (256, 19.3, 20.2), (512,
// 32.7, 20.8); at 100 x 300 x 8192: 8.3 and 36. There is no term for the output, and the
// model takes the slower side at 777 x 1000 x 1041 (narrow 13.1, pairs 9.9) and for 128 tokens
// through 11008 x 4096 (narrow 30.4, where 256 tokens take 20.8 in pairs).
TilePlan plan_tiles(int64_t T, int64_t R, int num_kb, bool one_scale, int sm_count) {
    auto ceil_div = [](int64_t p, int64_t q) { return (p + q - 1) / q; };
    TilePlan best{0, 1};
    const int64_t pair_waves = ceil_div(ceil_div(T, 256) * ceil_div(R, 256), std::max(1, sm_count / 2));
    double least = 4.0 + static_cast<double>(pair_waves) * num_kb * (one_scale ? 0.5 : 0.7);
    for (int bn : {16, 32, 64, 128}) {
        if (bn > 16 && bn / 2 >= T) break;  // the width below holds all tokens
        const int64_t tiles = ceil_div(R, kTileM) * ceil_div(T, bn);
        const int slots = sm_count * (bn <= 64 ? 2 : 1);
        for (int splits : {1, 2, 4, 8}) {
            if (splits > 1 && (splits > num_kb || tiles * splits > slots)) break;
            const int64_t kbs = ceil_div(num_kb, splits), waves = ceil_div(tiles * splits, slots);
            const double chain = static_cast<double>(waves * kbs) * (bn == 128 ? 0.45 : bn == 64 ? 0.30 : 0.25);
            const double loads = static_cast<double>(tiles * num_kb) * (kTileM + bn) * 128 / 7e6;
            const double t = 4.9 + std::max(chain, loads) + (splits == 8 ? 1.3 : splits > 1 ? 0.3 : 0.0);
            if (t < least) {
                least = t;
                best = TilePlan{bn, splits};
            }
        }
    }
    return best;
}

}  // namespace

void fp8_linear_plan(int64_t T, int64_t R, int64_t K, bool one_scale, int sm_count, int* tile_tokens, int* splits) {
    TilePlan plan{kMaxDecodeTokens, 1};
    if (!fp8_decode_serves(T)) plan = plan_tiles(T, R, static_cast<int>((K + 127) / 128), one_scale, sm_count);
    *tile_tokens = plan.bn;
    *splits = plan.splits;
}

cudaError_t take_fp8_linear_status(int* code, cudaStream_t stream) {
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

cudaError_t launch_fp8_linear(const void* xq, int64_t ld_x, bool x_e5m2, const ScaleView& xs, const void* wq,
                              int64_t ld_w, bool w_e5m2, const ScaleView& ws, int64_t T, int64_t R, int64_t K,
                              const void* bias, vnm_dtype bias_type, int act, void* y, int64_t ld_y, vnm_dtype y_type,
                              int* status, int skip_stage, int sm_count, cudaStream_t stream) {
    auto ceil_div = [](int64_t p, int64_t q) { return (p + q - 1) / q; };
    if (K > 0 && skip_stage < 0 && fp8_decode_serves(T))
        return launch_fp8_decode(xq, ld_x, x_e5m2, xs, wq, ld_w, w_e5m2, ws, T, R, K, bias, bias_type, act, y, ld_y,
                                 y_type, stream);
    const TilePlan plan = plan_tiles(T, R, static_cast<int>(ceil_div(K, 128)), ws.shift != 0, sm_count);
    const bool wide = plan.bn == 0;
    Fp8LinearArgs g{};
    if (wide)
        g = Fp8LinearArgs{xq, wq, ld_x, ld_w, x_e5m2, w_e5m2, xs, ws, T, R, K, ld_y, 1, false};
    else
        g = Fp8LinearArgs{wq, xq, ld_w, ld_x, w_e5m2, x_e5m2, ws, xs, R, T, K, 1, ld_y, true};
    FlArgs a{};
    a.m = g.m;
    a.n = g.n;
    a.num_kb = static_cast<int>(ceil_div(K, 128));
    a.ps = g.ps;
    a.qs = g.qs;
    auto quad = [](const ScaleView& v) { return v.cs == 1 && v.rs % 4 == 0 && reinterpret_cast<uintptr_t>(v.p) % 16 == 0; };
    a.quad_scales = quad(g.qs) && (!wide || quad(g.ps));  // (narrow tiles' P is not read through the ring)
    a.y = y;
    a.y_ms = g.y_ms;
    a.y_ns = g.y_ns;
    a.y_type = y_type;
    const uintptr_t elem = y_type == VNM_F32 ? 4 : 2;
    a.y_tma = (reinterpret_cast<uintptr_t>(y) | static_cast<uintptr_t>(ld_y) * elem) % 16 == 0;
    a.y_ends = static_cast<uintptr_t>(R) * elem % 16 == 0;
    a.bias = bias;
    a.bias_type = bias_type;
    a.bias_on_m = g.bias_on_m;
    a.act = act;
    a.status = status;
    a.skip_stage = skip_stage;
    if (K == 0) {
        const int64_t n = std::min<int64_t>(ceil_div(T * R, 256), 16 * sm_count);
        fp8_linear_empty_kernel<<<static_cast<unsigned>(n), 256, 0, stream>>>(a);
        return cudaGetLastError();
    }
    if (wide)
        return y_type == VNM_F32 ? ws.shift ? run<256, true, 2, true>(g, a, 1, sm_count, stream)
                                            : run<256, false, 2, true>(g, a, 1, sm_count, stream)
               : ws.shift        ? run<256, true, 2>(g, a, 1, sm_count, stream)
                                 : run<256, false, 2>(g, a, 1, sm_count, stream);
    switch (plan.bn) {
        case 16: return run<16, false, 1>(g, a, plan.splits, sm_count, stream);
        case 32: return run<32, false, 1>(g, a, plan.splits, sm_count, stream);
        case 64: return run<64, false, 1>(g, a, plan.splits, sm_count, stream);
        default: return run<128, false, 1>(g, a, plan.splits, sm_count, stream);
    }
}

}  // namespace vnm
