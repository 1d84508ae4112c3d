// Tensor-core (tcgen05 / TMEM / TMA) split-KV decode of the 8-bit latent cache
// (MLA_KV_MXFP8) of the DeepSeek-V3 shape: kv_lora_rank 512, rope 64, block size 64.
//
// The same decomposition as the bf16 kernel (mla_wide.cu): a pair of CTAs a stream and
// 128-row tile, CTA `half` owning latent output dims [256*half, 256*half + 256); a step is
// two cache blocks, 128 tokens; one step buffer of nine 16 KB column blocks ([128 tokens x
// 64 dims] bf16), the five that only the scores read (the other half's latent dims and the
// rope key) released before the four own ones; P over the scores in tensor memory.
//
// A code times a power of two is a bf16, so expanding the codes into the bf16 blocks is
// exact and everything after it is as over a bf16 cache of the same values. What differs:
//   expansion  eight warps read codes and scales into registers, 36 registers a step half
//              and thread, issued while the half before is worked on (so that the latency
//              of L2, about a thousand cycles, is never waited for), and write the swizzled
//              blocks, zeros for tokens past the end. The score-only blocks are expanded
//              while softmax and P . V of the step before run, the own ones while the score
//              MMAs over the score-only blocks do.
//   softmax    four warps, a thread a row of 128 scores, in two passes over tensor memory
//              (maximum; then weights, 32 columns at a time): no exchange between warps,
//              and few enough registers that 14 warps get 128 each. With 18 warps (eight of
//              softmax) a thread has 96, and the spilled ones, more than fit the L1 that is
//              left beside 227 KB of shared memory, came from L2 at every step.
// The rope key comes by TMA.
//
// Tensor memory: O [0,256), S / P [256,384), Q's own latent dims [384,512).
// Roles: warp 0 = rope keys (+ L2 prefetch of the codes); warp 1 = TMEM owner, lane 0
// issues every MMA; warps 4..7 = Q loads, softmax, epilogue (TMEM lanes 32*(w%4)..+31);
// warps 2, 3, 8..13 = expansion. Every wait is bounded (2 s); a wait that gives up records
// FLAG_TIMEOUT and the CTA winds down without trapping.
#include "mla_internal.cuh"
#include "mla_mx.cuh"
#include "mla_ptx.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>
#include <math_constants.h>
#include <string.h>

namespace mla {
namespace wmx {

using namespace ptx;

constexpr int kThreads = 448;
constexpr int kSoftmaxThreads = 128;                  // warps 4..7
constexpr int kExpandThreads = 256;                   // warps 2, 3, 8..13
constexpr int kTile = 64;                             // tokens per cache block
constexpr int kStep = 2 * kTile;                      // tokens per step (MMA N of the scores)
constexpr int kRows = 128;                            // query rows per CTA (MMA M)
constexpr int kD = 576;                               // r + d_R
constexpr int kBlocks = 9;                            // 64-dim column blocks per token row
constexpr uint32_t kBox = kTile * 128;                // [64 tokens x 64 dims] bf16: 8 KB
constexpr uint32_t kCol = kStep * 128;                // one column block of a step: 16 KB
constexpr uint32_t kQBlock = kRows * 128;             // [128 rows x 64 dims] bf16: 16 KB
constexpr int kQTmemBlocks = 4;                       // Q's own latent dims
constexpr int kQSmemBlocks = 5;                       // Q's score-only dims
constexpr uint32_t kOffBuf = 0;
constexpr uint32_t kOffQ = kOffBuf + kBlocks * kCol;          // 144 KB
constexpr uint32_t kOffBar = kOffQ + kQSmemBlocks * kQBlock;   // 224 KB
constexpr uint32_t kSmemBytes = kOffBar + 512 + 1024;          // + alignment slack
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr uint32_t kColO = 0, kColS = 256, kColQ = 384;
constexpr uint32_t kEpiBoxBytes = 32 * 128;           // epilogue box: [32 rows x 64 dims] bf16
static_assert(4 * 4 * kEpiBoxBytes <= kQSmemBlocks * kQBlock, "four boxes a warp");
constexpr unsigned long long kTimeoutNs = 2000000000ull;       // 2 s bounded-wait safety net
#ifndef MLA_MX_PREFETCH_AHEAD
#define MLA_MX_PREFETCH_AHEAD 4
#endif
constexpr int kPrefetchAhead = MLA_MX_PREFETCH_AHEAD;       // blocks prefetched into L2 ahead

// Column block of the step buffer that holds dims [64c, 64c + 64): own blocks are the
// latent blocks 4*half .. 4*half + 3; the five score-only blocks are the other half's
// latent blocks and the rope block (index 8).
__device__ __forceinline__ int score_only_block(int half, int k) { return k < 4 ? 4 * (1 - half) + k : 8; }

// Pipeline timestamps for performance analysis, compiled only with -DMLA_TRACE: clock64
// at each hand-off of one CTA (stream MLA_TRACE_STREAM, half MLA_TRACE_HALF, row tile 0)
// for its first kTraceSteps steps. Product builds contain none of it.
#ifdef MLA_TRACE
#ifndef MLA_TRACE_STREAM
#define MLA_TRACE_STREAM 0
#endif
#ifndef MLA_TRACE_HALF
#define MLA_TRACE_HALF 0
#endif
constexpr int kTraceSteps = 64;
__device__ long long g_mxtrace[16][kTraceSteps];
#define WTRACE(ev, step)                                                                                          \
    do {                                                                                                          \
        if (blockIdx.x == MLA_TRACE_HALF && blockIdx.y == 0 && blockIdx.z == MLA_TRACE_STREAM && (step) < kTraceSteps) \
            g_mxtrace[ev][step] = clock64();                                                                       \
    } while (0)
#else
#define WTRACE(ev, step) \
    do {                 \
    } while (0)
#endif
#define WTRACE_E(ev)                          \
    do {                                      \
        if (warp == 2 && lane == 0) WTRACE(ev, K); \
    } while (0)
// events: 0 score-only boxes issued, 1 own boxes issued (producer), 2 score-only blocks
// landed, 3 part 1 issued, 4 own blocks landed, 5 QK committed, 6 P seen, 7 PV issued
// (MMA), 8 S seen, 9 row max agreed, 10 P stored (softmax), 11 entry, 12 score-only blocks
// free, 13 expanded, 14 own blocks free, 15 expanded (warp 2 of the 8-bit kind)

struct Bars {
    uint64_t full_a;          // the step's score-only blocks are there
    uint64_t full_v;          // the step's own blocks are there
    uint64_t empty_a;         // the score MMAs over the score-only blocks completed
    uint64_t empty_v;         // PV of the step completed
    uint64_t s_full;
    uint64_t p_full;
    uint64_t pv_done;
    uint64_t q_stage;         // the staged tensor-memory part of Q landed in the Q region
    uint64_t q_smem;          // Q's shared-memory part landed in the Q region
    uint64_t q_tmem;          // the tensor-memory part of Q is stored
    uint64_t qreg_free;       // every softmax thread is done with the Q region
    uint64_t mma_fin;
    uint32_t tmem_base;
    int32_t abort_flag;
};
static_assert(sizeof(Bars) <= 512, "barriers must fit below the exchange area");

__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, Bars *bars, int32_t *status) {
    return mbar_wait_bounded(bar, parity, &bars->abort_flag, status, FLAG_TIMEOUT, kTimeoutNs);
}
__device__ __forceinline__ bool aborted(Bars *bars) { return *(volatile int32_t *)&bars->abort_flag != 0; }

// Physical block of logical block `lb` of sequence b, or -1.
__device__ __forceinline__ int block_of(const DecodeParams &p, int b, int lb) {
    if (lb >= p.max_blocks) return -1;
    const int blk = p.block_table[(size_t)b * p.max_blocks + lb];
    return (blk >= 0 && blk < p.s.num_blocks) ? blk : -1;
}

__host__ __device__ constexpr int steps_of(int t0, int t1) { return (t1 - t0 + kStep - 1) / kStep; }

__global__ void __launch_bounds__(kThreads, 1)
decode_mx_kernel(const __grid_constant__ CUtensorMap rope_map, const __grid_constant__ CUtensorMap q_map,
                 const __grid_constant__ CUtensorMap o_map, const DecodeParams p) {
    const int half = blockIdx.x;             // 0/1: which 256 latent output dims
    const int g = blockIdx.y;                // query row tile
    const int stream = blockIdx.z;           // work stream (persistent over its items)
    const int rows_seq = p.q_len * p.s.H;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    Bars *bars = (Bars *)(smem + kOffBar);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) WTRACE(11, 0);
    if (tid == 0) {
        mbar_init(&bars->full_a, 1 + kExpandThreads);
        mbar_init(&bars->full_v, kExpandThreads);
        mbar_init(&bars->empty_a, 1);
        mbar_init(&bars->empty_v, 1);
        mbar_init(&bars->s_full, 1);
        mbar_init(&bars->p_full, kSoftmaxThreads);
        mbar_init(&bars->pv_done, 1);
        mbar_init(&bars->q_stage, 1);
        mbar_init(&bars->q_smem, 1);
        mbar_init(&bars->q_tmem, kSoftmaxThreads);
        mbar_init(&bars->qreg_free, kSoftmaxThreads);
        mbar_init(&bars->mma_fin, 1);
        bars->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&bars->tmem_base)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    // Each CTA asks L2 for its share of the query (a call input; only a cache hint),
    // so that the first work item's query load does not wait on DRAM.
    if (tid == 0) {
        const size_t q_bytes = (size_t)p.B * rows_seq * kD * 2;
        const size_t n_ctas = (size_t)gridDim.x * gridDim.y * gridDim.z;
        const size_t cta = ((size_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
        const size_t share = ((q_bytes + n_ctas - 1) / n_ctas + 15) & ~(size_t)15;
        const size_t lo = cta * share;
        if (lo < q_bytes) {
            const size_t hi = min(q_bytes, lo + share);
            prefetch_l2((const uint8_t *)p.q + lo, (uint32_t)((hi - lo) & ~(size_t)15));
        }
    }
    // the set-up above overlaps the planner; its schedule is read only from here on.
    // The combine may launch from here: the planner has completed, so the combine can
    // read the schedule's split ranges before its own wait.
    pdl_wait();
    pdl_trigger();
    const int i0 = p.stream_start[stream], i1 = p.stream_start[stream + 1];
    if (i0 >= i1) {                          // no work for this stream (CTA-uniform)
        if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
        return;
    }

    if (warp == 0) {
        // ================================================= rope keys (+ L2 prefetch)
        // The warp runs converged; one lane per box.
        const bool prefetcher = kPrefetchAhead > 0 && half == 0 && g == 0;
        int pi = i0, pt = 0, ahead = 0;
        auto advance_prefetch = [&]() {
            while (pi < i1 && ahead < kPrefetchAhead) {
                const WorkItem it = p.work[pi];
                const int nt = (it.t1 - it.t0 + kTile - 1) / kTile;
                if (pt >= nt) { ++pi; pt = 0; continue; }
                const int blk = block_of(p, it.b, it.t0 / kTile + pt);
                if (blk >= 0) {
                    prefetch_l2(p.codes + (size_t)blk * (kTile * 512), kTile * 512);
                    prefetch_l2(p.mx_scale + (size_t)blk * (kTile * 16), kTile * 16);
                    prefetch_l2(p.rope + (size_t)blk * (kTile * 64), kTile * 128);
                }
                ++pt;
                ++ahead;
            }
        };
        const int oob_row = p.s.num_blocks * kTile;   // past the end: TMA fills zeros
        int K = 0;
        bool ok = true;
        for (int i = i0; i < i1 && ok; ++i) {
            const WorkItem it = p.work[i];
            const int nt = (it.t1 - it.t0 + kTile - 1) / kTile;
            const int ns = steps_of(it.t0, it.t1);
            for (int j = 0; j < ns; ++j, ++K) {
                // lane u < 2: tile u of the step (a missing or bad block reads zeros past the
                // end; the softmax marks a bad block's rows NaN)
                int row0 = oob_row;
                if (lane < 2 && 2 * j + lane < nt) {
                    const int blk = block_of(p, it.b, it.t0 / kTile + 2 * j + lane);
                    if (blk >= 0) row0 = blk * kTile;
                    else raise_flag(p.status, FLAG_BAD_BLOCK);
                }
                // the rope block is free once the previous step's score MMAs over it completed
                if (K > 0 && !__all_sync(0xffffffffu, mbar_wait(&bars->empty_a, (K - 1) & 1, bars, p.status))) {
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_expect_tx(&bars->full_a, 2 * kBox);
                __syncwarp();
                if (lane < 2) tma_load_2d(smem + kOffBuf + 8 * kCol + lane * kBox, &rope_map, 0, row0, &bars->full_a);
                if (lane == 0 && prefetcher) {
                    ahead = max(0, ahead - 2);
                    advance_prefetch();
                }
            }
        }
        // drain: never leave a copy in flight into this CTA's shared memory (the barrier also
        // counts the expanding warps, which arrive unless the CTA aborts; bounded)
        if (K > 0) mbar_drain(&bars->full_a, (K - 1) & 1);
        __syncwarp();
    } else if (warp == 1) {
        // ================================================= MMA issuer: lane 0 alone
        if (lane == 0) {
            constexpr uint32_t kIdQk = idesc_bf16(128, 128, false);
            constexpr uint32_t kIdPv = idesc_bf16(128, 256, true);
            const uint32_t qt = tmem + kColQ, d_s = tmem + kColS, d_o = tmem + kColO;
            uint64_t qd = sdesc(smem_u32(smem + kOffQ), 16, 1024);
            uint64_t bd = sdesc(smem_u32(smem + kOffBuf), 16, 1024);
            // MN-major V: 64-dim atoms 16 KB apart (column blocks), 8-token groups 1 KB apart
            uint64_t vd = sdesc(smem_u32(smem + kOffBuf + 4 * half * kCol), kCol, 1024);
            bool ok = true;
            int K = 0;
            int item_no = 0;
            for (int i = i0; i < i1 && ok; ++i, ++item_no) {
                const WorkItem it = p.work[i];
                const int ns = steps_of(it.t0, it.t1);
                if (!mbar_wait(&bars->q_tmem, item_no & 1, bars, p.status)) { ok = false; break; }
                for (int j = 0; j < ns; ++j, ++K) {
                    // opaque: the descriptors of 44 MMAs are formed when they are used, not kept
                    asm volatile("" : "+l"(qd), "+l"(bd), "+l"(vd));
                    if (!mbar_wait(&bars->full_a, K & 1, bars, p.status)) { ok = false; break; }
                    WTRACE(2, K);
                    // S / P's tensor memory is free once the previous step's PV completed
                    if (K > 0 && !mbar_wait(&bars->pv_done, (K - 1) & 1, bars, p.status)) { ok = false; break; }
                    // the item's first step: Q's shared-memory part may still be landing
                    if (j == 0 && !mbar_wait(&bars->q_smem, item_no & 1, bars, p.status)) { ok = false; break; }
                    tc_fence_after();
                    // part 1: score-only blocks, Q from shared memory. K-step (k, s): Q slot k /
                    // column block score_only_block(k), 32-byte step s inside the swizzle atom
                    // (descriptor start addresses advance in 16-byte units)
#pragma unroll
                    for (int k = 0; k < kQSmemBlocks; ++k) {
                        const uint32_t cb = (uint32_t)score_only_block(half, k) * kCol;
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            const uint64_t a = qd + (uint64_t)((k * kQBlock + 32 * s) >> 4);
                            const uint64_t b = bd + (uint64_t)((cb + 32 * s) >> 4);
                            if (k == 0 && s == 0) mma_ss_k<kIdQk, 0>(d_s, a, b);
                            else mma_ss_k<kIdQk, 1>(d_s, a, b);
                        }
                    }
                    mma_commit(&bars->empty_a);
                    WTRACE(3, K);
                    if (!mbar_wait(&bars->full_v, K & 1, bars, p.status)) { ok = false; break; }
                    WTRACE(4, K);
                    tc_fence_after();
                    // part 2: own blocks, Q from tensor memory (8 columns per K-step)
#pragma unroll
                    for (int k = 0; k < kQTmemBlocks; ++k) {
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            mma_ts_k<kIdQk, 1>(d_s, qt + 32 * k + 8 * s,
                                               bd + (uint64_t)(((4 * half + k) * kCol + 32 * s) >> 4));
                    }
                    mma_commit(&bars->s_full);
                    WTRACE(5, K);
                    // PV once the softmax stored P
                    if (!mbar_wait(&bars->p_full, K & 1, bars, p.status)) { ok = false; break; }
                    WTRACE(6, K);
                    tc_fence_after();
                    // K-step kk: P columns 8 kk (two bf16 tokens per column), V rows 16 kk
                    // (two 8-token groups, 2 KB)
#pragma unroll
                    for (int kk = 0; kk < kStep / 16; ++kk) {
                        if (kk == 0 && j == 0) mma_ts_k<kIdPv, 0>(d_o, d_s, vd);
                        else mma_ts_k<kIdPv, 1>(d_o, d_s + 8 * kk, vd + (uint64_t)(128 * kk));
                    }
                    mma_commit(&bars->pv_done);
                    mma_commit(&bars->empty_v);
                    WTRACE(7, K);
                }
            }
            mma_commit(&bars->mma_fin);
            mbar_wait(&bars->mma_fin, 0, bars, p.status);
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        // ================================================= Q loads, softmax, epilogue
        // Thread (warp w, lane) owns query row 32*(w%4) + lane. Every branch around tcgen05.ld
        // / tcgen05.st is warp-uniform.
        //
        // The Q region serves three uses in turn: staging the tensor-memory part of an
        // item's Q (TMA in, tcgen05.st out), the epilogue's output boxes, and Q's
        // shared-memory part that the score MMAs read. qreg_free completes once every
        // softmax thread is done with a staging or epilogue use; the TMA issuer (warp 4
        // lane 0) waits for it before loading into the region.
        const int wq = warp & 3;
        const int row = 32 * wq + lane;
        const int row_seq = g * kRows + row;
        const bool row_valid = row_seq < rows_seq;
        const bool issuer = warp == 4 && lane == 0;
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * wq) << 16);
        const uint32_t tS = lane_addr + kColS;
        bool ok = true;
        int K = 0, uses = 0, nstage = 0;
        // TMA of Q part `round` of work item `item` into the Q region (issuer only): round
        // 0 stages the tensor-memory part (the own latent blocks), round 1 loads the
        // shared-memory part (the score-only dims, in score_only_block order).
        auto issue_q = [&](int item, int round) -> bool {
            if (!issuer) return true;
            if (uses > 0 && !mbar_wait(&bars->qreg_free, (uses - 1) & 1, bars, p.status)) return false;
            const int qrow = p.work[item].b * rows_seq + g * kRows;
            if (round == 0) {
                mbar_expect_tx(&bars->q_stage, kQTmemBlocks * kQBlock);
                for (int k = 0; k < kQTmemBlocks; ++k)
                    tma_load_2d(smem + kOffQ + k * kQBlock, &q_map, 64 * (4 * half + k), qrow, &bars->q_stage);
            } else {
                mbar_expect_tx(&bars->q_smem, kQSmemBlocks * kQBlock);
                for (int k = 0; k < kQSmemBlocks; ++k)
                    tma_load_2d(smem + kOffQ + k * kQBlock, &q_map, 64 * score_only_block(half, k), qrow, &bars->q_smem);
            }
            return true;
        };
        // Staged Q -> tensor memory, a thread its row.
        auto load_q_tmem = [&]() -> bool {
            if (!__all_sync(0xffffffffu, mbar_wait(&bars->q_stage, nstage & 1, bars, p.status))) return false;
            ++nstage;
#pragma unroll 1
            for (int k = 0; k < kQTmemBlocks; ++k) {
                uint32_t v[32];
                const uint8_t *blk = smem + kOffQ + k * kQBlock;
#pragma unroll
                for (int ch = 0; ch < 8; ++ch) {
                    const uint4 u = *(const uint4 *)(blk + sw128(row, ch));
                    v[4 * ch + 0] = u.x;
                    v[4 * ch + 1] = u.y;
                    v[4 * ch + 2] = u.z;
                    v[4 * ch + 3] = u.w;
                }
                TMEM_ST32(lane_addr + kColQ + 32 * k, v);
            }
            mbar_arrive(&bars->qreg_free);
            ++uses;
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&bars->q_tmem);
            return true;
        };
        ok = __all_sync(0xffffffffu, issue_q(i0, 0));
        ok = ok && load_q_tmem();
        ok = ok && __all_sync(0xffffffffu, issue_q(i0, 1));
        // Scores stay unscaled where the scale is positive: the row max then commutes with
        // the scaling and each exponent argument is one fma.
        const bool pos_scale = p.scale_log2 > 0.f;
        const float cs = pos_scale ? p.scale_log2 : 1.f;
        for (int i = i0; i < i1 && ok; ++i) {
            const WorkItem it = p.work[i];
            const int L = p.seq_lens[it.b];
            const int t0 = it.t0, t1 = it.t1;
            const int nt = (t1 - t0 + kTile - 1) / kTile;
            const int ns = steps_of(t0, t1);
            const int last_vis = L - p.q_len + (row_valid ? row_seq / p.s.H : 0);
            float m_used = -CUDART_INF_F, l = 0.f;
            bool bad_item = false;
            for (int t = 0; t < nt; ++t) bad_item |= block_of(p, it.b, t0 / kTile + t) < 0;
            for (int j = 0; j < ns && ok; ++j, ++K) {
                if (!__all_sync(0xffffffffu, mbar_wait(&bars->s_full, K & 1, bars, p.status))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (tid == 128) WTRACE(8, K);
                const int n_vis = row_valid ? max(0, min(t1, last_vis + 1) - (t0 + j * kStep)) : 0;
                const bool plain = pos_scale && __all_sync(0xffffffffu, n_vis >= kStep);
                // hidden slots -> -inf
                auto mask = [&](uint32_t (&sv)[32], int c) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float v = pos_scale ? __uint_as_float(sv[e]) : __uint_as_float(sv[e]) * p.scale_log2;
                        sv[e] = __float_as_uint(32 * c + e < n_vis ? v : -CUDART_INF_F);
                    }
                };
                float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
                auto max_of = [&](uint32_t (&sv)[32], int c) {
                    if (!plain) mask(sv, c);
#pragma unroll
                    for (int e = 0; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(sv[e]));
                };
                // (loops of two chunks, not unrolled: with every role's code laid out straight the
                // warps waited for instructions more than for anything else)
                uint32_t s0[32], s1[32];
                TMEM_LD32(tS, s0);
#pragma unroll 1
                for (int c = 0; c < 4; c += 2) {
                    tmem_wait_ld(s0);
                    TMEM_LD32(tS + 32 * c + 32, s1);
                    max_of(s0, c);
                    tmem_wait_ld(s1);
                    TMEM_LD32(tS + ((32 * c + 64) & 127), s0);     // at the end chunk 0 again
                    max_of(s1, c + 1);
                }
                const float m_new = fmaxf(m_used, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * cs);
                if (tid == 128) WTRACE(9, K);
                float alpha = 1.f;
                bool rescale = false;
                if (m_new > m_used + 8.f) {
                    alpha = exp2f(m_used - m_new);        // 0 when nothing was accumulated yet
                    m_used = m_new;
                    rescale = j > 0;
                }
                const float nmb = m_used == -CUDART_INF_F ? -CUDART_INF_F : -m_used;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                // weights of columns 32 c .. 32 c + 31, in place (16 registers), over the first
                // columns of chunk c / 2, which have been read
                auto weights = [&](uint32_t (&sv)[32], int c) {
                    if (!plain) mask(sv, c);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float a = ex2(fmaf(__uint_as_float(sv[2 * e]), cs, nmb));
                        const float b = ex2(fmaf(__uint_as_float(sv[2 * e + 1]), cs, nmb));
                        const __nv_bfloat162 hh = __floats2bfloat162_rn(a, b);
                        sv[e] = *(const uint32_t *)&hh;
                        sum[(2 * e) & 3] += a;     // fp32 row sum: the LSE does not see the rounding of P
                        sum[(2 * e + 1) & 3] += b;
                    }
                    TMEM_ST16(tS + 16 * c, sv);
                };
#pragma unroll 1
                for (int c = 0; c < 4; c += 2) {
                    tmem_wait_ld(s0);
                    TMEM_LD32(tS + 32 * c + 32, s1);
                    weights(s0, c);
                    tmem_wait_ld(s1);
                    if (c == 0) TMEM_LD32(tS + 64, s0);
                    weights(s1, c + 1);
                }
                l = l * alpha + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
                // O *= alpha: the previous step's PV completed before these scores were
                // computed (the MMA thread issues a step's score MMAs after it)
                if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        TMEM_LD32(lane_addr + kColO + 32 * c, s0);
                        tmem_wait_ld(s0);
#pragma unroll
                        for (int k = 0; k < 32; ++k) s0[k] = __float_as_uint(__uint_as_float(s0[k]) * alpha);
                        TMEM_ST32(lane_addr + kColO + 32 * c, s0);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bars->p_full);
                if (tid == 128) WTRACE(10, K);
            }
            // ---- end of this item. The Q region is free (the item's last score MMAs have
            // completed): stage the next item's tensor-memory Q while the last PV runs, then
            // write this item's output through the region, then load the next item's
            // shared-memory Q part.
            const bool have_next = i + 1 < i1;
            if (ok && have_next) ok = __all_sync(0xffffffffu, issue_q(i + 1, 0));
            if (ok && ns > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bars->pv_done, (K - 1) & 1, bars, p.status));
            tc_fence_after();
            if (ok && have_next) ok = load_q_tmem();
            if (ok && have_next)
                ok = __all_sync(0xffffffffu, mbar_wait(&bars->qreg_free, (uses - 1) & 1, bars, p.status));
            const bool bad = aborted(bars) || !ok || bad_item;
            // Epilogue: O / l -> partial slot i, rounded to bf16; [32 rows x 64 dims] boxes
            // (128B-swizzled) through the region, one TMA store each; rows past the
            // sequence's rows are clipped by the tensor map.
            if (ok) {
                const float inv = l > 0.f ? 1.f / l : 0.f;
                const uint64_t keep = l2_policy_evict_last();
                uint8_t *boxes = smem + kOffQ + 4 * wq * kEpiBoxBytes;
                const int y = g * kRows + 32 * wq;
                const bool store = y < rows_seq;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint8_t *box = boxes + c * kEpiBoxBytes;
#pragma unroll 1
                    for (int hh = 0; hh < 2; ++hh) {
                        uint32_t ov[32];
                        TMEM_LD32(lane_addr + kColO + 64 * c + 32 * hh, ov);
                        tmem_wait_ld(ov);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t pk4[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __nv_bfloat162 h2 = __floats2bfloat162_rn(
                                    __uint_as_float(ov[8 * q + 2 * e]) * inv, __uint_as_float(ov[8 * q + 2 * e + 1]) * inv);
                                pk4[e] = *(const uint32_t *)&h2;
                            }
                            *(uint4 *)(box + sw128(lane, 4 * hh + q)) = make_uint4(pk4[0], pk4[1], pk4[2], pk4[3]);
                        }
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0 && store) {
                        tma_store_3d_hint(&o_map, box, 256 * half + 64 * c, y, i, keep);
                        bulk_commit();
                    }
                }
                if (lane == 0) bulk_wait_read();
                __syncwarp();
            }
            mbar_arrive(&bars->qreg_free);
            ++uses;
            if (row_valid && half == 0)
                p.part_lse[(size_t)i * rows_seq + row_seq] =
                    bad ? CUDART_NAN_F : (l > 0.f ? m_used + log2f(l) : -CUDART_INF_F);
            tc_fence_before();     // O reads complete before the next item's first PV
            if (ok && have_next) ok = __all_sync(0xffffffffu, issue_q(i + 1, 1));
        }
        if (lane == 0) bulk_wait_all();   // this warp's output stores have landed
    } else {
        // ================================================= expansion of the codes
        // Warp e takes rows 8 e .. 8 e + 7 of both tiles, four rows and a 128-byte line of
        // each (two 64-dim column blocks) at a time. Eight lanes take 16 codes each: four of
        // one row's first block and four of the neighbouring row's second, so that their
        // 16-byte stores fall on eight different swizzled chunks.
        const int e = warp < 4 ? warp - 2 : warp - 6, p8 = lane & 7;
        const bool second = p8 >= 4;
        const int r4 = (lane >> 3) ^ (second ? 1 : 0);
        // a lane's first chunk and the shared address of its row of the first 8-row atom
        const uint32_t chunk = (uint32_t)((2 * (p8 & 3)) ^ r4) << 4;
        const uint32_t to0 = smem_u32(smem + kOffBuf) + (second ? kCol : 0u) + 1024u * e + 128u * r4;
        struct Half {                      // of a step: the score-only or the own dims
            uint4 c[2][2][2];              // [tile][row group][column block pair]
            uint2 s[2][2];                 // the row's eight scales of these dims
        };
        struct Step {
            int row0[2], valid[2];         // token row of each tile's first slot; its tokens
        };
        auto step_at = [&](const WorkItem &it, int L, int j) {
            Step st;
            const int nt = (it.t1 - it.t0 + kTile - 1) / kTile;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int t = 2 * j + u;
                const int blk = t < nt ? block_of(p, it.b, it.t0 / kTile + t) : -1;
                st.row0[u] = blk * kTile;
                st.valid[u] = blk >= 0 ? min(kTile, L - (it.t0 + t * kTile)) : 0;
            }
            return st;
        };
        auto load = [&](Half &x, const Step &st, int cb) {     // column blocks cb .. cb + 3
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int row = 8 * e + 4 * q + r4;
                    x.s[u][q] = make_uint2(0, 0);
                    x.c[u][q][0] = x.c[u][q][1] = make_uint4(0, 0, 0, 0);    // zeros for slots past the end
                    if (row < st.valid[u]) {
                        const size_t tok = (size_t)(st.row0[u] + row);
                        const uint8_t *src = p.codes + tok * 512 + 64 * cb + 16 * p8;
#pragma unroll
                        for (int w = 0; w < 2; ++w)
                            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(x.c[u][q][w].x), "=r"(x.c[u][q][w].y), "=r"(x.c[u][q][w].z), "=r"(x.c[u][q][w].w)
                                         : "l"(src + 128 * w));
                        asm volatile("ld.global.v2.u32 {%0, %1}, [%2];"
                                     : "=r"(x.s[u][q].x), "=r"(x.s[u][q].y)
                                     : "l"(p.mx_scale + tok * 16 + 2 * cb));
                    }
                }
        };
        auto expand = [&](const Half &x, int cb) {
            // scales up to 1 take one multiplication
            const uint32_t any = x.s[0][0].x | x.s[0][0].y | x.s[0][1].x | x.s[0][1].y | x.s[1][0].x | x.s[1][0].y |
                                 x.s[1][1].x | x.s[1][1].y;
            const bool small = !__any_sync(0xffffffffu, any & 0x80808080u);
            const uint32_t to = to0 + (uint32_t)cb * kCol;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const uint32_t sw = w ? x.s[u][q].y : x.s[u][q].x;
                        uint4 o0, o1;
                        if (small) mx_expand16(x.c[u][q][w], mx_scale120(sw, p8 >> 1), o0, o1);
                        else mx_expand16(x.c[u][q][w], kMx2p120, mx_scale_bf162((sw >> (8 * (p8 >> 1))) & 0xffu), o0, o1);
                        // row 4 q + r4 of the atom flips bit 2 of the chunk with q
                        const uint32_t at = to + (chunk ^ (64u * q)) + 512u * q + 8192u * u + 2u * w * kCol;
                        const uint32_t at1 = to + (chunk ^ (64u * q) ^ 16u) + 512u * q + 8192u * u + 2u * w * kCol;
                        st_shared16(at, o0);
                        st_shared16(at1, o1);
                    }
        };
        const int cb_a = 4 * (1 - half), cb_v = 4 * half;
        // The steps in turn; false at the end.
        int i = i0, j = -1;
        WorkItem it = p.work[i];
        int L = p.seq_lens[it.b], ns = steps_of(it.t0, it.t1);
        auto next = [&](Step &st) {
            if (++j == ns) {
                j = 0;
                if (++i >= i1) return false;
                it = p.work[i];
                L = p.seq_lens[it.b];
                ns = steps_of(it.t0, it.t1);
            }
            st = step_at(it, L, j);
            return true;
        };
        // Turn K: step K's own dims, then step K + 1's score-only ones, then the loads for the next
        // turn, all at once: they have the time until the next P . V is done to arrive (a
        // load issued shortly before a batch is used holds that up, too: loads share the few
        // counters that a use waits for).
        Step s0, s1, s2;                   // of K, K + 1, K + 2
        Half x, a;                         // own dims of K, score-only ones of K + 1
        bool more = next(s0);
        load(x, s0, cb_a);
        // turn -1 is step 0's score-only part; one copy of the expansion for both parts
        for (int K = -1;; ++K) {
            bool ok = true;
#pragma unroll 1
            for (int part = K < 0 ? 1 : 0; part < 2 && ok; ++part) {
                uint64_t *free_bar = part ? &bars->empty_a : &bars->empty_v;
                const int use = part ? K : K - 1;              // the step that used the blocks before
                if (use >= 0 && !__all_sync(0xffffffffu, mbar_wait(free_bar, use & 1, bars, p.status))) {
                    ok = false;
                    break;
                }
                WTRACE_E(part ? 12 : 14);
                expand(x, part ? cb_a : cb_v);
                fence_proxy_async();
                mbar_arrive(part ? &bars->full_a : &bars->full_v);
                WTRACE_E(part ? 13 : 15);
                if (part == 0) {
                    if (!more) ok = false;                     // no step K + 1
                    else x = a;
                }
            }
            if (!ok) break;
            if (K < 0) s1 = s0;
            load(x, s1, cb_v);
            more = next(s2);
            if (more) load(a, s2, cb_a);
            s1 = s2;
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// ---------------------------------------------------------------- host side
static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = (PFN_cuTensorMapEncodeTiled_v12000)ptr;
    }
    return fn;
}

// 2-D bf16 map over a row-major [rows, cols] matrix, 128-byte swizzled boxes of
// [box_rows, 64]. Rows past the end read as zero.
static bool make_map(CUtensorMap *map, const void *base, uint64_t rows, uint32_t box_rows, uint64_t cols) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
    cuuint32_t box[2] = {64, box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

// 3-D bf16 map over the partial outputs [slots, rows_seq, r], boxes of [32 rows x 64
// dims] with the 128-byte swizzle (stores clip rows >= rows_seq).
static bool make_out_map(CUtensorMap *map, void *base, int r, int rows_seq, int slots) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)r, (cuuint64_t)rows_seq, (cuuint64_t)slots};
    cuuint64_t strides[2] = {(cuuint64_t)r * 2, (cuuint64_t)rows_seq * r * 2};
    cuuint32_t box[3] = {64, 32, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult res = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, estr,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return res == CUDA_SUCCESS;
}

}  // namespace wmx

cudaError_t launch_decode_mx(const DecodeParams &p, int32_t max_work, cudaStream_t st) {
    const int rows_seq = p.q_len * p.s.H;
    CUtensorMap rope_map, q_map, o_map;
    if (!wmx::make_map(&rope_map, p.rope, (uint64_t)p.s.num_blocks * p.s.bs, wmx::kTile, (uint64_t)p.s.dR) ||
        !wmx::make_map(&q_map, p.q, (uint64_t)p.B * rows_seq, wmx::kRows, wmx::kD) ||
        !wmx::make_out_map(&o_map, p.part_o, p.s.r, rows_seq, max_work))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(wmx::decode_mx_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)wmx::kSmemBytes);
    if (e != cudaSuccess) return e;
    dim3 grid(2, (rows_seq + wmx::kRows - 1) / wmx::kRows, p.streams);
    return launch_pdl(wmx::decode_mx_kernel, grid, dim3(wmx::kThreads), wmx::kSmemBytes, st, rope_map, q_map, o_map, p);
}

}  // namespace mla

#ifdef MLA_TRACE
extern "C" int mla_mx_trace_read(long long *events) {
    return (int)cudaMemcpyFromSymbol(events, mla::wmx::g_mxtrace, sizeof(mla::wmx::g_mxtrace));
}
#endif
