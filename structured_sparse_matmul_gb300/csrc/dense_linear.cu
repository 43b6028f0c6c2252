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
// dense_pair_kernel, many tokens: pairs of CTAs (cta_group::2), 256 rows of X by 256 of W
// a tile (each CTA loads its own 128 rows of X and 128 of W; of a gated pair, the
// first CTA loads Wg's and the second Wu's rows, and a tile is 128 features of
// both), persistent, two TMEM accumulators of 256 columns, so that a tile's
// epilogue runs under the next one's MMAs.
//   warp 0     TMA producer: stages of 64 elements of K, 128B swizzle.
//   warp 1     TMEM owner, MMA issuer (one thread of the first CTA).
//   warps 4..  epilogue: 32 rows x 128 columns of the tile a warp, by way of shared
//              memory (fp32), from which 8 neighbouring columns go to a lane: whole
//              16-byte loads of the residual and stores of Y.
//
// dense_narrow_kernel, few tokens or few tiles: W on the MMA's M side (its rows fill the
// tensor cores' rows), 16 to 128 tokens a tile, K over the CTAs of a cluster,
// which add their sums up through distributed shared memory in rank order.
//
// The tensor cores' fp32 sums truncate: over K they lose about K * 2^-30 of
// random sums and six times that of sums of one sign (measured: 9e-6 and 5e-5 at
// K = 8192). Nothing next to a rounding to 16 bits, but it is to fp32 outputs, so
// for those the sums are taken out every kChunk elements of K and added in registers.
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
constexpr int kChunk = 2048 / kBlockK;
constexpr int kMaxSplits = 8;
constexpr int kMaxDevicesDl = 64;
constexpr int kGroupM = 8;

struct Maps {
    CUtensorMap x[2], w[2];
};

struct GemmArgs {
    OutArgs o;
    int kind;
    int num_kb;       // K blocks of one product
    int total_kb;     // of an output's sum
    int chunk_kb;     // K blocks of one TMEM sum
    int x_tiles;      // tiles of X's rows, of one product
    int m_tiles, n_tiles, tiles;
    int splits, kb_per_split;
    bool x_t, w_t;
    uint32_t idesc;
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
__device__ __forceinline__ void st_shared_f4(uint32_t addr, float a, float b, float c, float d) {
    st_shared_v4(addr, __float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
}

// ------------------------------------------------------------------ pairs of CTAs

constexpr int kPairStages = 5;
constexpr int kPairStageBytes = 2 * kOperandBytes;
constexpr int kPairHelpers = 4, kPairEpilogue = 8;
constexpr int kPairThreads = 32 * (kPairHelpers + kPairEpilogue);
constexpr int kBoxBytes = 8192;  // a warp's staged sums: 32 rows x 64 columns (gated: 32 of each)
constexpr int kPairSmem = kPairStages * kPairStageBytes + kPairEpilogue * kBoxBytes + 1024;
static_assert(kPairSmem > 116 * 1024 && kPairSmem <= 226 * 1024, "one CTA an SM: each holds all of its TMEM");
// Registers of the variant that adds chunks up (128 sums a thread), in warps:
// 4 x 56 + 8 x 224 = 12 x 168 of the launch.
constexpr int kSumLaunchRegs = 168, kSumHelperRegs = 56, kSumAddRegs = 224;
static_assert(kPairHelpers * kSumHelperRegs + kPairEpilogue * kSumAddRegs == (kPairHelpers + kPairEpilogue) * kSumLaunchRegs,
              "register shares");

// 16-byte piece j of row `row` of a staged box of `pitch` bytes a row.
__device__ __forceinline__ uint32_t piece(uint32_t buf, int pitch, int row, int j) {
    return buf + row * pitch + 16 * (j ^ (row & 7));
}

// Rows m0 .. m0 + 31, columns n0 .. n0 + 63 of Y from their staged sums.
__device__ __forceinline__ void finish_rows(const OutArgs& o, int seg, uint32_t buf, int64_t m0, int64_t n0, int lane) {
    const int c = lane & 7, top = lane >> 3;  // columns 8c .., rows top, top + 4, ...
    const int64_t n = n0 + 8 * c, left = o.R - n;
    if (o.bias != nullptr || o.act != VNM_ACT_NONE) {
        float b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = o.bias != nullptr && j < left ? load_any(o.bias, o.bias_type, n + j) : 0.f;
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            const uint32_t p0 = piece(buf, 256, 4 * i + top, 2 * c), p1 = piece(buf, 256, 4 * i + top, 2 * c + 1);
            const float4 x = ld_shared_v4(p0), y = ld_shared_v4(p1);
            float v[8] = {x.x + b[0], x.y + b[1], x.z + b[2], x.w + b[3], y.x + b[4], y.y + b[5], y.z + b[6], y.w + b[7]};
            activate8(o.act, v);
            st_shared_f4(p0, v[0], v[1], v[2], v[3]);  // (read again by this lane alone)
            st_shared_f4(p1, v[4], v[5], v[6], v[7]);
        }
    }
    if (left <= 0) return;
    void* const y = o.y[seg];
    const void* const res = o.res[seg];
#pragma unroll 1
    for (int i = 0; i < 8; i += 4) {
        float r[4][8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t m = m0 + 4 * (i + k) + top;
            if (res != nullptr && m < o.T) load8(res, o.y_type, m * o.ld_res + n, o.res_vec, left, r[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int row = 4 * (i + k) + top;
            const int64_t m = m0 + row;
            if (m >= o.T) break;
            const float4 p = ld_shared_v4(piece(buf, 256, row, 2 * c)), q = ld_shared_v4(piece(buf, 256, row, 2 * c + 1));
            float v[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
            if (res != nullptr) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += r[k][j];
            }
            store8(y, o.y_type, m * o.ld_y + n, o.y_vec, left, v);
        }
    }
}

template <bool GATED, bool SUM>
__global__ void __launch_bounds__(kPairThreads, 1)
    dense_pair_kernel(const __grid_constant__ Maps maps, const __grid_constant__ GemmArgs a) {
    constexpr int ST = kPairStages;
    constexpr int kTileN = GATED ? 128 : 256;  // columns of Y of a tile
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[ST];   // the stage has landed in both CTAs (the first CTA's)
    __shared__ __align__(8) uint64_t empty_bar[ST];  // its MMAs are done
    __shared__ __align__(8) uint64_t accf_bar[2];    // the TMEM sum is complete
    __shared__ __align__(8) uint64_t acce_bar[2];    // and has been read by both CTAs (the first CTA's)
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x & 1);
    const int tile0 = static_cast<int>(blockIdx.x >> 1), tile_step = static_cast<int>(gridDim.x >> 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(smem_u32(&full_bar[s]), 1);
            mbar_init(smem_u32(&empty_bar[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&accf_bar[s]), 1);
            mbar_init(smem_u32(&acce_bar[s]), 2 * kPairEpilogue);
        }
        abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc_group<2>(smem_u32(&tmem_slot), 512);
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers and TMEM exist
    tc_fence_after_sync();
    const uint32_t tmem = tmem_slot;
    volatile int* abort = &abort_flag;

    if (SUM && warp < kPairHelpers) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kSumHelperRegs));
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
            const int wrow = GATED ? nt * kTile : nt * 256 + rank * kTile;
            for (int kb = 0; kb < a.total_kb; ++kb, ++it) {
                if (!mbar_wait_warp(smem_u32(&empty_bar[slot]), phase, abort)) {
                    run = false;
                    break;
                }
                if (elect_one() && (it != a.skip_stage || blockIdx.x != 0)) {
                    const bool second = kb >= a.num_kb;  // of a sum of two
                    const CUtensorMap* tx = &maps.x[second || seg];
                    const CUtensorMap* tw = &maps.w[GATED ? rank : second];
                    const int k = (second ? kb - a.num_kb : kb) * kBlockK;
                    const uint32_t sx = smem_base + slot * kPairStageBytes, sw = sx + kOperandBytes;
                    const uint32_t fb = smem_u32(&full_bar[slot]), lead = dsmem_map(fb, 0);
                    // the second CTA's bytes may arrive before the first CTA expects them: the
                    // phase cannot end before that CTA's own arrival
                    if (rank == 0) mbar_arrive_expect_tx(fb, 2 * kPairStageBytes);
                    if (a.x_t) {
                        tma_load_2d_pair(sx, tx, xrow, k, lead);
                        tma_load_2d_pair(sx + 8192, tx, xrow + 64, k, lead);
                    } else {
                        tma_load_2d_pair(sx, tx, k, xrow, lead);
                    }
                    if (a.w_t) {
                        tma_load_2d_pair(sw, tw, wrow, k, lead);
                        tma_load_2d_pair(sw + 8192, tw, wrow + 64, k, lead);
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
            for (int kb0 = 0; kb0 < a.total_kb && run; kb0 += a.chunk_kb) {
                const int kb1 = min(a.total_kb, kb0 + a.chunk_kb);
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
                        const uint64_t off = static_cast<uint64_t>((slot * kPairStageBytes) >> 4);
#pragma unroll
                        for (uint32_t s = 0; s < 4; ++s)
                            tc_mma_f16_pair(tmem + acc * 256, xdesc + off + s * xstep, wdesc + off + s * wstep, a.idesc,
                                            kb > kb0 || s > 0 ? 1u : 0u);
                        tc_commit_group<2>(smem_u32(&empty_bar[slot]));
                        if (kb + 1 == kb1) tc_commit_group<2>(smem_u32(&accf_bar[acc]));
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
        if (SUM) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumAddRegs));
        const int quarter = warp & 3, half = (warp - kPairHelpers) >> 2;  // TMEM lanes 32 quarter ..; columns
        const uint32_t lane_addr = static_cast<uint32_t>(32 * quarter) << 16;
        const uint32_t acce_lead = dsmem_map(smem_u32(&acce_bar[0]), 0);
        const uint32_t buf = smem_base + ST * kPairStageBytes + (warp - kPairHelpers) * kBoxBytes;
        int acc = 0;
        uint32_t acc_phase = 0;
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
        // 32 of the lane's sums from column j of a staged row of 256 bytes on
        auto stage32 = [&](const uint32_t (&v)[32], int j) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                st_shared_v4(piece(buf, 256, lane, j + u), v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
        };
        for (int tile = tile0; tile < a.tiles && run; tile += tile_step) {
            int mt, nt;
            tile_at(a, tile, mt, nt);
            const int seg = a.kind == kTwoByRows && mt >= a.x_tiles ? 1 : 0;
            const int64_t m0 = static_cast<int64_t>((mt - seg * a.x_tiles) * 2 + rank) * kTile + 32 * quarter;
            const int64_t n0 = static_cast<int64_t>(nt) * kTileN + half * (kTileN / 2);
            if constexpr (SUM) {
                float sum[128];
#pragma unroll
                for (int c = 0; c < 128; ++c) sum[c] = 0.f;
                for (int kb0 = 0; kb0 < a.total_kb; kb0 += a.chunk_kb) {
                    if (!wait_sum()) break;
#pragma unroll
                    for (int c = 0; c < 128; c += 32) {
                        uint32_t v[32];
                        tmem_ld(tmem + lane_addr + acc * 256 + half * 128 + c, v);
                        tmem_wait_ld(v);
#pragma unroll
                        for (int j = 0; j < 32; ++j) sum[c + j] += __uint_as_float(v[j]);
                    }
                    release();
                }
                if (!run) break;
#pragma unroll
                for (int c = 0; c < 128; c += 64) {
#pragma unroll
                    for (int u = 0; u < 16; ++u)
                        st_shared_f4(piece(buf, 256, lane, u), sum[c + 4 * u], sum[c + 4 * u + 1], sum[c + 4 * u + 2],
                                     sum[c + 4 * u + 3]);
                    __syncwarp();
                    finish_rows(a.o, seg, buf, m0, n0 + c, lane);
                    __syncwarp();
                }
            } else if constexpr (GATED) {
                if (!wait_sum()) break;
                const uint32_t taddr = tmem + lane_addr + acc * 256;
                const int64_t m = m0 + lane;
                float gs = 1.f, ginv = 1.f, us = 1.f, uinv = 1.f;
                if (a.o.keep == kKeep8) {
                    // the row's largest magnitudes over the tile's 128 columns, a group of the 8-bit
                    // form (columns past the edge are zeros); both halves read them all
                    float top[2] = {0.f, 0.f};
#pragma unroll 1
                    for (int c = 0; c < 256; c += 32) {
                        uint32_t v[32];
                        tmem_ld(taddr + c, v);
                        tmem_wait_ld(v);
                        float t = c < 128 ? top[0] : top[1];
#pragma unroll
                        for (int j = 0; j < 32; ++j) t = max_magnitude(t, __uint_as_float(v[j]));
                        if (c < 128)
                            top[0] = t;
                        else
                            top[1] = t;
                    }
                    gs = group_scale(top[0], a.o.e5m2, ginv);
                    us = group_scale(top[1], a.o.e5m2, uinv);
                    if (half == 0 && m < a.o.T) {
                        a.o.g.s[m * a.o.g.s_rs + nt * a.o.g.s_cs] = gs;
                        a.o.u.s[m * a.o.u.s_rs + nt * a.o.u.s_cs] = us;
                    }
                }
#pragma unroll 1
                for (int c = 0; c < 64; c += 32) {
                    uint32_t v[32];
                    tmem_ld(taddr + half * 64 + c, v);
                    tmem_wait_ld(v);
                    stage32(v, 0);
                    tmem_ld(taddr + 128 + half * 64 + c, v);
                    tmem_wait_ld(v);
                    stage32(v, 8);
                    if (c + 32 == 64) release();
                    __syncwarp();
                    const int q = lane & 3, first = lane >> 2;  // features 8q .., rows first, first + 8, ...
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        const int row = 8 * i + first;
                        const float4 p0 = ld_shared_v4(piece(buf, 256, row, 2 * q)), p1 = ld_shared_v4(piece(buf, 256, row, 2 * q + 1));
                        const float4 q0 = ld_shared_v4(piece(buf, 256, row, 8 + 2 * q)),
                                     q1 = ld_shared_v4(piece(buf, 256, row, 9 + 2 * q));
                        float g[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
                        const float u[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
                        const float rgs = __shfl_sync(0xFFFFFFFFu, gs, row), rgi = __shfl_sync(0xFFFFFFFFu, ginv, row);
                        const float rus = __shfl_sync(0xFFFFFFFFu, us, row), rui = __shfl_sync(0xFFFFFFFFu, uinv, row);
                        if (m0 + row < a.o.T) finish_gated8(a.o, m0 + row, n0 + c + 8 * q, g, u, rgs, rgi, rus, rui);
                    }
                    __syncwarp();
                }
            } else {
                if (!wait_sum()) break;
                const uint32_t taddr = tmem + lane_addr + acc * 256 + half * 128;
#pragma unroll 1
                for (int c = 0; c < 128; c += 64) {
                    uint32_t v[32];
                    tmem_ld(taddr + c, v);
                    tmem_wait_ld(v);
                    stage32(v, 0);
                    tmem_ld(taddr + c + 32, v);
                    tmem_wait_ld(v);
                    stage32(v, 8);
                    if (c + 64 == 128) release();
                    __syncwarp();
                    finish_rows(a.o, seg, buf, m0, n0 + c, lane);
                    __syncwarp();
                }
            }
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();  // neither CTA leaves while the other's arrivals or MMAs may reach it
    if (threadIdx.x == 0 && abort_flag) record_error(a.status ? a.status : g_status, VNM_ERR_TIMEOUT, 13);
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_group<2>(tmem, 512);
    }
}

// ------------------------------------------------------------------ narrow tiles

template <int BN, bool GATED>
struct NarrowCfg {
    static constexpr int kWBytes = (GATED ? 2 : 1) * kOperandBytes;
    static constexpr int kStageBytes = kWBytes + BN * 128;
    // two CTAs an SM, whose waits overlap, where their rings are deep enough
    static constexpr int kCtas = GATED && BN >= 64 ? 1 : 2;
    static constexpr int kStages = GATED ? (BN >= 128 ? 4 : BN == 64 ? 5 : 3) : BN == 128 ? 3 : BN == 64 ? 4 : 5;
    static constexpr int kTmemCols = 2 * BN;  // two sums: of g and of u, or of two chunks
    static constexpr int kThreads = 192;
    static constexpr int kSmem = kStages * kStageBytes + 1024;
    static constexpr int kPartBytes = (GATED ? 2 : 1) * kTile * BN * 4;
    static_assert(kPartBytes <= kStages * kStageBytes, "the CTA's sums fit the stage ring");
    static_assert(kCtas == 2 ? 2 * (kSmem + 2048) <= 228 * 1024 : kSmem > 116 * 1024 && kSmem <= 226 * 1024, "shared memory");
    static_assert(kCtas * kTmemCols <= 512 && kTmemCols >= 32, "TMEM of the CTAs that share an SM");
};

template <int BN, bool GATED>
__global__ void __launch_bounds__(NarrowCfg<BN, GATED>::kThreads, NarrowCfg<BN, GATED>::kCtas)
    dense_narrow_kernel(const __grid_constant__ Maps maps, const __grid_constant__ GemmArgs a) {
    using Cfg = NarrowCfg<BN, GATED>;
    constexpr int ST = Cfg::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full_bar[ST], empty_bar[ST];
    __shared__ __align__(8) uint64_t accf_bar[2], acce_bar[2];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    float* const part = reinterpret_cast<float*>(smem_raw + (smem_base - smem_u32(smem_raw)));  // [g, u][BN][kTile], over the ring
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x) % a.splits, tile = static_cast<int>(blockIdx.x) / a.splits;
    // tiles of tokens fastest: the CTAs that run together share W's tiles
    const int mt = tile / a.n_tiles, nt = tile - mt * a.n_tiles;
    const int seg = a.kind == kTwoByRows && nt >= a.x_tiles ? 1 : 0;
    const int xrow = (nt - seg * a.x_tiles) * BN, wrow = mt * kTile;
    const int kb0 = rank * a.kb_per_split, kb1 = max(kb0, min(a.total_kb, kb0 + a.kb_per_split));

    // one stage's loads into its slot
    auto load_stage = [&](int slot, int kb) {
        const uint32_t fb = smem_u32(&full_bar[slot]), sw = smem_base + slot * Cfg::kStageBytes, sx = sw + Cfg::kWBytes;
        const bool second = kb >= a.num_kb;  // of a sum of two
        const CUtensorMap* tx = &maps.x[second || seg];
        const int k = (second ? kb - a.num_kb : kb) * kBlockK;
        mbar_arrive_expect_tx(fb, Cfg::kStageBytes);
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); ++h) {
            const CUtensorMap* tw = &maps.w[GATED ? h : second];
            const uint32_t to = sw + h * kOperandBytes;
            if (a.w_t) {
                tma_load_2d(to, tw, wrow, k, fb);
                tma_load_2d(to + 8192, tw, wrow + 64, k, fb);
            } else {
                tma_load_2d(to, tw, k, wrow, fb);
            }
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
        for (int k = 0; k < early; ++k)
            if (k != a.skip_stage || blockIdx.x != 0) load_stage(k, kb0 + k);
    }
    if (warp == 1) tmem_alloc_group<1>(smem_u32(&tmem_slot), Cfg::kTmemCols);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
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
        const uint64_t wdesc = operand_desc(smem_base, a.w_t), xdesc = operand_desc(smem_base + Cfg::kWBytes, a.x_t);
        const uint32_t wstep = operand_step(a.w_t), xstep = operand_step(a.x_t);
        int it = 0, slot = 0, chunk = 0;
        uint32_t phase = 0;
        bool run = true;
        for (int c0 = kb0; c0 < kb1 && run; c0 += a.chunk_kb, ++chunk) {
            const int c1 = min(kb1, c0 + a.chunk_kb), acc = GATED ? 0 : chunk & 1;
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
                    for (uint32_t s = 0; s < 4; ++s) {
                        const uint32_t more = kb > c0 || s > 0 ? 1u : 0u;
                        tc_mma_f16(tmem + acc * BN, wdesc + off + s * wstep, xdesc + off + s * xstep, a.idesc, more);
                        if (GATED)
                            tc_mma_f16(tmem + BN, wdesc + off + (kOperandBytes >> 4) + s * wstep, xdesc + off + s * xstep, a.idesc,
                                       more);
                    }
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
        if constexpr (GATED) {
            const bool any = kb0 < kb1;
            if (!any || mbar_wait_warp(smem_u32(&accf_bar[0]), 0, abort)) {
                tc_fence_after_sync();
#pragma unroll 1
                for (int c = 0; c < 2 * BN; c += LD) {
                    uint32_t v[LD];
                    if (any) {
                        tmem_ld(tmem + lane_addr + c, v);
                        tmem_wait_ld(v);
                    }
#pragma unroll
                    for (int j = 0; j < LD; ++j) part[(c + j) * kTile + row] = any ? __uint_as_float(v[j]) : 0.f;
                }
            }
        } else {
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
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_group<1>(tmem, Cfg::kTmemCols);
    }
    if (a.splits > 1) cluster_sync_all();
    // add the cluster's sums, in rank order, each CTA a share of the tokens; 16 lanes x 8 features a token
    const int share = (BN + a.splits - 1) / a.splits, c0 = rank * share, c1 = min(BN, c0 + share);
    const OutArgs& o = a.o;
    const int64_t r = static_cast<int64_t>(wrow) + 8 * (lane & 15), left = o.R - r;
    float bias[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) bias[j] = !GATED && o.bias != nullptr && j < left ? load_any(o.bias, o.bias_type, r + j) : 0.f;
#pragma unroll 1
    for (int base = c0 + 2 * warp; base < c1; base += 2 * (Cfg::kThreads / 32)) {
        const int c = base + (lane >> 4);
        const int64_t t = static_cast<int64_t>(xrow) + c;
        const bool here = c < c1 && t < o.T;
        float v[GATED ? 2 : 1][8];
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); ++h) {
            const uint32_t addr = smem_base + 4 * ((h * BN + min(c, BN - 1)) * kTile + 8 * (lane & 15));
#pragma unroll
            for (int j = 0; j < 8; ++j) v[h][j] = 0.f;
#pragma unroll
            for (int s = 0; s < kMaxSplits; ++s) {
                if (s >= a.splits) break;
                const uint32_t from = a.splits > 1 ? dsmem_map(addr, s) : addr;
                const float4 p = a.splits > 1 ? dsmem_ld_v4(from) : ld_shared_v4(from);
                const float4 q = a.splits > 1 ? dsmem_ld_v4(from + 16) : ld_shared_v4(from + 16);
                v[h][0] += p.x, v[h][1] += p.y, v[h][2] += p.z, v[h][3] += p.w;
                v[h][4] += q.x, v[h][5] += q.y, v[h][6] += q.z, v[h][7] += q.w;
            }
        }
        if constexpr (GATED) {
            float scale[2] = {1.f, 1.f}, inv[2] = {1.f, 1.f};
            if (o.keep == kKeep8) {
                // the tile's 128 features are a group of the 8-bit form (past the edge they are zeros)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float top = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) top = max_magnitude(top, v[h][j]);
#pragma unroll
                    for (int d = 8; d > 0; d >>= 1) top = max_magnitude(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                    scale[h] = group_scale(top, o.e5m2, inv[h]);
                }
                if (here && (lane & 15) == 0) {
                    o.g.s[t * o.g.s_rs + mt * o.g.s_cs] = scale[0];
                    o.u.s[t * o.u.s_rs + mt * o.u.s_cs] = scale[1];
                }
            }
            if (here) finish_gated8(o, t, r, v[0], v[1], scale[0], inv[0], scale[1], inv[1]);
        } else if (here && left > 0) {
            float res[8];
            if (o.res[seg] != nullptr) load8(o.res[seg], o.y_type, t * o.ld_res + r, o.res_vec, left, res);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[0][j] += bias[j];
            activate8(o.act, v[0]);
            if (o.res[seg] != nullptr) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[0][j] += res[j];
            }
            store8(o.y[seg], o.y_type, t * o.ld_y + r, o.y_vec, left, v[0]);
        }
    }
    if (a.splits > 1) cluster_sync_all();  // no CTA leaves while others read its sums
    if (threadIdx.x == 0 && abort_flag) record_error(a.status ? a.status : g_status, VNM_ERR_TIMEOUT, 14);
}

// K = 0: the sums are 0.
__global__ void dense_empty_kernel(const OutArgs o, int kind) {
    const int64_t per_row = (o.R + 7) / 8;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < o.T * per_row;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t t = i / per_row, r = 8 * (i - t * per_row), left = o.R - r;
        if (kind == kGatedPair) {
            float g[8] = {}, u[8] = {};
            if (o.keep == kKeep8 && r % 128 == 0) {
                o.g.s[t * o.g.s_rs + (r / 128) * o.g.s_cs] = kMinScale;
                o.u.s[t * o.u.s_rs + (r / 128) * o.u.s_cs] = kMinScale;
            }
            finish_gated8(o, t, r, g, u, kMinScale, 1.f / kMinScale, kMinScale, 1.f / kMinScale);
            continue;
        }
        for (int seg = 0; seg < (kind == kTwoByRows ? 2 : 1); ++seg) {
            float v[8], res[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = o.bias != nullptr && j < left ? load_any(o.bias, o.bias_type, r + j) : 0.f;
            activate8(o.act, v);
            if (o.res[seg] != nullptr) {
                load8(o.res[seg], o.y_type, t * o.ld_res + r, o.res_vec, left, res);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += res[j];
            }
            store8(o.y[seg], o.y_type, t * o.ld_y + r, o.y_vec, left, v);
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

template <typename Kernel>
cudaError_t launch(Kernel kernel, int64_t ctas, int threads, int smem, int cluster, const Maps& maps, const GemmArgs& a,
                   cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(cluster);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, maps, a);
}

template <bool GATED, bool SUM>
cudaError_t run_pair(const ProductArgs& p, GemmArgs a, int sm_count, cudaStream_t stream) {
    static std::atomic<bool> set[kMaxDevicesDl];
    a.x_tiles = static_cast<int>(ceil_div(p.T, 2 * kTile));
    a.m_tiles = a.x_tiles * (p.kind == kTwoByRows ? 2 : 1);
    a.n_tiles = static_cast<int>(ceil_div(p.R, GATED ? kTile : 2 * kTile));
    const int64_t tiles = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    a.tiles = static_cast<int>(tiles);
    a.splits = 1;
    a.kb_per_split = a.total_kb;
    a.idesc = f16_idesc(2 * kTile, 256, p.bf16, a.x_t, a.w_t);
    Maps maps;
    if (!encode_all(&maps, p, kTile, kTile)) return cudaErrorInvalidValue;
    const cudaError_t e = prepare(dense_pair_kernel<GATED, SUM>, kPairSmem, SUM ? kSumLaunchRegs : 0, set);
    if (e != cudaSuccess) return e;
    return launch(dense_pair_kernel<GATED, SUM>, 2 * std::min<int64_t>(tiles, std::max(1, sm_count / 2)), kPairThreads, kPairSmem, 2,
                  maps, a, stream);
}

template <int BN, bool GATED>
cudaError_t run_narrow(const ProductArgs& p, GemmArgs a, int splits, cudaStream_t stream) {
    using Cfg = NarrowCfg<BN, GATED>;
    static std::atomic<bool> set[kMaxDevicesDl];
    a.x_tiles = static_cast<int>(ceil_div(p.T, BN));
    a.n_tiles = a.x_tiles * (p.kind == kTwoByRows ? 2 : 1);
    a.m_tiles = static_cast<int>(ceil_div(p.R, kTile));
    const int64_t tiles = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
    if (tiles * splits > INT32_MAX) return cudaErrorInvalidValue;
    a.tiles = static_cast<int>(tiles);
    a.splits = splits;
    a.kb_per_split = static_cast<int>(ceil_div(a.total_kb, splits));
    a.idesc = f16_idesc(kTile, BN, p.bf16, a.w_t, a.x_t);
    Maps maps;
    if (!encode_all(&maps, p, BN, kTile)) return cudaErrorInvalidValue;
    const cudaError_t e = prepare(dense_narrow_kernel<BN, GATED>, Cfg::kSmem, 0, set);
    if (e != cudaSuccess) return e;
    return launch(dense_narrow_kernel<BN, GATED>, tiles * splits, Cfg::kThreads, Cfg::kSmem, splits, maps, a, stream);
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

struct TilePlan {
    int bn, splits;
};

// The times the plan compares, in us: a launch with its first loads and its last stores; then the
// longer of a CTA's chain of K blocks and of its tiles' loads from L2.
TilePlan plan_tiles(const ProductArgs& p, int sm_count) {
    const bool gated = p.kind == kGatedPair, two = p.kind == kTwoByRows;
    const int num_kb = static_cast<int>(ceil_div(p.K, kBlockK)) * (p.kind == kSumOfTwo ? 2 : 1);
    TilePlan best{0, 1};
    const int64_t pair_tiles = ceil_div(p.T, 256) * (two ? 2 : 1) * ceil_div(p.R, gated ? 128 : 256);
    double least = 5.0 + static_cast<double>(ceil_div(pair_tiles, std::max(1, sm_count / 2))) * num_kb * 0.3;
    for (int bn : {16, 32, 64, 128}) {
        if (bn > 16 && bn / 2 >= p.T && !(p.x[0].transposed && bn <= 64)) break;  // the width below holds all tokens
        if (p.x[0].transposed && bn < 64) continue;  // (a box of transposed X is 64 tokens)
        const int64_t tiles = ceil_div(p.R, kTile) * ceil_div(p.T, bn) * (two ? 2 : 1);
        const int slots = sm_count * (gated && bn >= 64 ? 1 : 2);
        for (int splits : {1, 2, 4, 8}) {
            if (splits > 1 && (splits > num_kb || tiles * splits > slots)) break;
            const int64_t kbs = ceil_div(num_kb, splits), waves = ceil_div(tiles * splits, slots);
            const double chain = static_cast<double>(waves * kbs) * (bn == 128 ? 0.40 : bn == 64 ? 0.30 : 0.25) * (gated ? 1.6 : 1.0);
            const double loads = static_cast<double>(tiles * num_kb) * (kTile * (gated ? 2 : 1) + bn) * 128 / 7e6;
            const double t = 4.9 + std::max(chain, loads) + (splits == 8 ? 1.3 : splits > 1 ? 0.3 : 0.0);
            if (t < least) {
                least = t;
                best = TilePlan{bn, splits};
            }
        }
    }
    return best;
}

bool few_tokens(const ProductArgs& p) {
    return p.T <= kFewTokens && (p.kind == kOneProduct || p.kind == kGatedPair) && p.keep == kKeepNone && !p.x[0].transposed &&
           !p.w[0].transposed;
}

}  // namespace

void product_plan(const ProductArgs& p, int sm_count, int* tile_tokens, int* splits) {
    TilePlan plan{kFewTokens, 1};
    if (!few_tokens(p)) plan = plan_tiles(p, sm_count);
    *tile_tokens = plan.bn;
    *splits = plan.splits;
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

cudaError_t launch_product(const ProductArgs& p, int sm_count, cudaStream_t stream) {
    if (p.K > 0 && p.skip_stage < 0 && few_tokens(p)) return launch_few_tokens(p, stream);
    GemmArgs a{};
    OutArgs& o = a.o;
    auto rows_aligned = [](const void* q, int64_t ld_bytes, int n) {
        return reinterpret_cast<uintptr_t>(q) % n == 0 && ld_bytes % n == 0;
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
    o.g_vec = rows_aligned(p.g.p, p.g.ld * k, 8 * k);
    o.u_vec = rows_aligned(p.u.p, p.u.ld * k, 8 * k);
    if (p.K == 0) {
        const int64_t n = std::min<int64_t>(ceil_div(p.T * ceil_div(p.R, 8), 256), 16 * sm_count);
        dense_empty_kernel<<<static_cast<unsigned>(n), 256, 0, stream>>>(o, p.kind);
        return cudaGetLastError();
    }
    a.kind = p.kind;
    a.num_kb = static_cast<int>(ceil_div(p.K, kBlockK));
    a.total_kb = a.num_kb * (p.kind == kSumOfTwo ? 2 : 1);
    a.chunk_kb = p.y_type == VNM_F32 ? kChunk : a.total_kb;
    a.x_t = p.x[0].transposed;
    a.w_t = p.w[0].transposed;
    a.status = p.status;
    a.skip_stage = p.skip_stage;
    const bool gated = p.kind == kGatedPair;
    const TilePlan plan = plan_tiles(p, sm_count);
    if (plan.bn == 0)
        return gated                  ? run_pair<true, false>(p, a, sm_count, stream)
               : p.y_type == VNM_F32 ? run_pair<false, true>(p, a, sm_count, stream)
                                     : run_pair<false, false>(p, a, sm_count, stream);
    return gated ? run_narrow<true>(plan.bn, p, a, plan.splits, stream) : run_narrow<false>(plan.bn, p, a, plan.splits, stream);
}

}  // namespace vnm
