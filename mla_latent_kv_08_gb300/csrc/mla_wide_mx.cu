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
// exact and everything after it is as over a bf16 cache of the same values. The rope key
// comes by TMA; the latent blocks are written by eight warps, which read codes and scales
// into registers, a part of a step (score-only or own dims) ahead of the one they expand.
// The score-only blocks are expanded while the softmax and P . V of the step before run,
// the own ones while the score MMAs over the score-only blocks do.
//
// Twenty warps leave a thread 96 registers; the split after launch (64 / 128 / 80) keeps
// every role out of local memory, whose spills, more than fit the L1 that 227 KB of shared
// memory leave, came from L2 at every step. With the roles' code laid out straight the
// warps waited for instruction fetches more than for anything else (3.9 warps an issue
// slot), so the expansion is one loop body for all parts.
//
// Measured, 32 sequences of 1024 to 8192 tokens (156k in all), 128 heads: 76 us, of which
// the codes' bytes at the copy rate are 15 us and the products at the cuBLAS rate 23 us;
// 16 sequences of 4096 to 32768 tokens with 8 drafts: 780 us against 272 us of products.
// The tensor pipe is busy for 39 % of the time. What bounds it is the chain of a step, one
// buffer deep: expand, score, softmax, P . V, and the scores that both CTAs of a pair make.
//
// Tensor memory: O [0,256), S / P [256,384), Q's other half of the latent dims [384,512).
// Roles: warp 0 = rope keys (+ L2 prefetch of the codes); warp 1 = TMEM owner, lane 0
// issues every MMA; warps 4..11 = Q loads, softmax, epilogue (TMEM lanes 32*(w%4)..+31);
// warps 12..19 = expansion. Every wait is bounded (2 s); a wait that gives up records
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

constexpr int kThreads = 640;
constexpr int kSoftmaxThreads = 256;                  // warps 4..11
constexpr int kExpandThreads = 256;                   // warps 12..19
// Registers a thread of the warpgroups (0: copies and MMA; 1, 2: softmax; 3, 4: expansion)
// once they are split again: what the launch had, 5 x 96.
constexpr int kRegsLaunch = 96, kRegsIssue = 64, kRegsSoftmax = 128, kRegsExpand = 80;
static_assert(kRegsIssue + 2 * kRegsSoftmax + 2 * kRegsExpand <= 5 * kRegsLaunch, "register split");
template <int N> __device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
constexpr int kTile = 64;                             // tokens per cache block
constexpr int kStep = 2 * kTile;                      // tokens per step (MMA N of the scores)
constexpr int kRows = 128;                            // query rows per CTA (MMA M)
constexpr int kD = 576;                               // r + d_R
constexpr int kBlocks = 9;                            // 64-dim column blocks per token row
constexpr uint32_t kBox = kTile * 128;                // [64 tokens x 64 dims] bf16: 8 KB
constexpr uint32_t kCol = kStep * 128;                // one column block of a step: 16 KB
constexpr uint32_t kQBlock = kRows * 128;             // [128 rows x 64 dims] bf16: 16 KB
constexpr int kQTmemBlocks = 4;                       // Q's other half of the latent dims
constexpr int kQSmemBlocks = 5;                       // Q's own latent dims, rope dims
constexpr uint32_t kOffBuf = 0;
constexpr uint32_t kOffQ = kOffBuf + kBlocks * kCol;          // 144 KB
constexpr uint32_t kOffBar = kOffQ + kQSmemBlocks * kQBlock;   // 224 KB
constexpr uint32_t kOffXchg = kOffBar + 512;                   // [2][128] fp32 row values
constexpr uint32_t kOffNan = kOffXchg + 1024;                  // int32 [128], see Bars::nan_step
constexpr uint32_t kSmemBytes = kOffNan + 512 + 1024;          // + alignment slack
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr uint32_t kColO = 0, kColS = 256, kColQ = 384;
constexpr uint32_t kEpiBoxBytes = 32 * 128;           // epilogue box: [32 rows x 64 dims] bf16
constexpr int kEpiBoxes = (int)((kQSmemBlocks * kQBlock) / (8 * kEpiBoxBytes));   // per warp at a time
static_assert(kEpiBoxes >= 1 && 2 % kEpiBoxes == 0, "epilogue boxes");
constexpr unsigned long long kTimeoutNs = 2000000000ull;       // 2 s bounded-wait safety net
constexpr int kPrefetchAhead = 4;                     // blocks prefetched into L2 ahead

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
        if (warp == 12 && lane == 0) WTRACE(ev, K); \
    } while (0)
// events: 2 score-only blocks there, 3 part 1 issued, 4 own blocks there, 5 QK committed, 6 P
// seen, 7 PV issued (MMA), 8 S seen, 9 row max agreed, 10 P stored (softmax), 11 entry, 12
// score-only blocks free, 13 expanded, 14 own blocks free, 15 expanded (warp 12)

struct Bars {
    uint64_t full_a;          // the step's score-only blocks are there
    uint64_t full_v;          // the step's own blocks are there
    uint64_t empty_a;         // the score MMAs over the score-only blocks completed
    uint64_t empty_v[2];      // PV over the step's first and second 64 tokens completed
    uint64_t s_full;
    uint64_t p_full;
    uint64_t pv_done;
    uint64_t q_stage;         // the staged tensor-memory part of Q landed in the Q region
    uint64_t q_smem;          // Q's shared-memory part landed in the Q region
    uint64_t q_tmem;          // the tensor-memory part of Q is stored
    uint64_t qreg_free;       // every softmax thread is done with the Q region
    uint64_t mma_fin;
    uint64_t xchg_full[4];    // lane quarter q: both halves of its rows wrote their value
    uint64_t xchg_read[4];    // lane quarter q: both halves read the other's value
    uint32_t tmem_base;
    int32_t abort_flag;
    // 1 + the last step with own dims that are not a number (a group's scale, or a code). They
    // are expanded to zeros (their product with a hidden row's weight 0 stays 0); the scores of
    // the tokens at kOffNan that hold this step become NaN for the rows that see them.
    int32_t nan_step;
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
        mbar_init(&bars->empty_v[0], 1);
        mbar_init(&bars->empty_v[1], 1);
        mbar_init(&bars->s_full, 1);
        mbar_init(&bars->p_full, kSoftmaxThreads);
        mbar_init(&bars->pv_done, 1);
        mbar_init(&bars->q_stage, 1);
        mbar_init(&bars->q_smem, 1);
        mbar_init(&bars->q_tmem, kSoftmaxThreads);
        mbar_init(&bars->qreg_free, kSoftmaxThreads);
        mbar_init(&bars->mma_fin, 1);
        for (int q = 0; q < 4; ++q) {
            mbar_init(&bars->xchg_full[q], 64);
            mbar_init(&bars->xchg_read[q], 64);
        }
        bars->abort_flag = 0;
        bars->nan_step = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    if (tid < kStep) ((int32_t *)(smem + kOffNan))[tid] = 0;
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
        reg_dec<kRegsIssue>();
        // The warp runs converged; one lane per box.
        // Only where several row tiles read the codes: one tile's own loads, a step ahead, are
        // early enough (a call of 32 sequences, 156k tokens: 87.8 us with, 86.2 without; 8 drafts
        // over 233k tokens 782 with, 788 without).
        const bool prefetcher = half == 0 && g == 0 && rows_seq > kRows;
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
        reg_dec<kRegsIssue>();
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
                    // part 1: score-only blocks; the latent ones with Q from tensor memory (8
                    // columns per K-step), so that the products take half of the shared memory's
                    // bandwidth while the own blocks are written (descriptor start addresses
                    // advance in 16-byte units)
#pragma unroll
                    for (int k = 0; k < kQTmemBlocks; ++k) {
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            const uint64_t b = bd + (uint64_t)(((4 * (1 - half) + k) * kCol + 32 * s) >> 4);
                            if (k == 0 && s == 0) mma_ts_k<kIdQk, 0>(d_s, qt, b);
                            else mma_ts_k<kIdQk, 1>(d_s, qt + 32 * k + 8 * s, b);
                        }
                    }
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        mma_ss_k<kIdQk, 1>(d_s, qd + (uint64_t)((4 * kQBlock + 32 * s) >> 4), bd + (uint64_t)((8 * kCol + 32 * s) >> 4));
                    mma_commit(&bars->empty_a);
                    WTRACE(3, K);
                    if (!mbar_wait(&bars->full_v, K & 1, bars, p.status)) { ok = false; break; }
                    WTRACE(4, K);
                    tc_fence_after();
                    // part 2: own blocks, Q from shared memory
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            mma_ss_k<kIdQk, 1>(d_s, qd + (uint64_t)((k * kQBlock + 32 * s) >> 4),
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
                        // the first tile's rows are written again while the second's are read
                        if (kk == kTile / 16 - 1) mma_commit(&bars->empty_v[0]);
                    }
                    mma_commit(&bars->pv_done);
                    mma_commit(&bars->empty_v[1]);
                    WTRACE(7, K);
                }
            }
            mma_commit(&bars->mma_fin);
            mbar_wait(&bars->mma_fin, 0, bars, p.status);
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 12) {
        // ================================================= Q loads, softmax, epilogue
        reg_inc<kRegsSoftmax>();
        // Warp w owns rows 32*(w%4)..+31 (its TMEM lane quarter) and half hs = (w-4)/4 of
        // the step: score columns 64*hs..+63 (tile hs), P columns 32*hs..+31, output
        // columns 128*hs..+127. Every branch around tcgen05.ld / tcgen05.st is warp-uniform.
        //
        // The Q region serves three uses in turn: staging the tensor-memory part of an
        // item's Q (TMA in, tcgen05.st out), the epilogue's output boxes, and Q's
        // shared-memory part that the score MMAs read. qreg_free completes once every
        // softmax thread is done with a staging or epilogue use; the TMA issuer (warp 4
        // lane 0) waits for it before loading into the region.
        const int wq = warp & 3;
        const int hs = (warp - 4) >> 2;
        const int row = 32 * wq + lane;
        const int row_seq = g * kRows + row;
        const bool row_valid = row_seq < rows_seq;
        const bool issuer = warp == 4 && lane == 0;
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * wq) << 16);
        float *xchg = (float *)(smem + kOffXchg);
        bool ok = true;
        int K = 0, nx = 0, uses = 0, nstage = 0;
        // Swap one value per row with the other half of the row (bounded waits). The
        // tensor-memory fences order each side's tcgen05 accesses before the swap against
        // the other side's after it.
        auto exchange = [&](float v, float &other) -> bool {
            if (nx > 0 && !mbar_wait(&bars->xchg_read[wq], (nx - 1) & 1, bars, p.status)) return false;
            xchg[hs * 128 + row] = v;
            tc_fence_before();
            mbar_arrive(&bars->xchg_full[wq]);
            if (!mbar_wait(&bars->xchg_full[wq], nx & 1, bars, p.status)) return false;
            tc_fence_after();
            other = xchg[(hs ^ 1) * 128 + row];
            mbar_arrive(&bars->xchg_read[wq]);
            ++nx;
            return true;
        };
        // TMA of Q part `round` of work item `item` into the Q region (issuer only): round
        // 0 stages the tensor-memory part (the other half's latent blocks), round 1 loads the
        // shared-memory part (the own latent blocks, then the rope block).
        auto issue_q = [&](int item, int round) -> bool {
            if (!issuer) return true;
            if (uses > 0 && !mbar_wait(&bars->qreg_free, (uses - 1) & 1, bars, p.status)) return false;
            const int qrow = p.work[item].b * rows_seq + g * kRows;
            if (round == 0) {
                mbar_expect_tx(&bars->q_stage, kQTmemBlocks * kQBlock);
                for (int k = 0; k < kQTmemBlocks; ++k)
                    tma_load_2d(smem + kOffQ + k * kQBlock, &q_map, 64 * (4 * (1 - half) + k), qrow, &bars->q_stage);
            } else {
                mbar_expect_tx(&bars->q_smem, kQSmemBlocks * kQBlock);
                for (int k = 0; k < kQSmemBlocks; ++k)
                    tma_load_2d(smem + kOffQ + k * kQBlock, &q_map, 64 * (k < 4 ? 4 * half + k : 8), qrow, &bars->q_smem);
            }
            return true;
        };
        // Staged Q -> tensor memory: thread (row, hs) moves blocks hs and hs + 2.
        auto load_q_tmem = [&]() -> bool {
            if (!__all_sync(0xffffffffu, mbar_wait(&bars->q_stage, nstage & 1, bars, p.status))) return false;
            ++nstage;
#pragma unroll 1
            for (int k = hs; k < kQTmemBlocks; k += 2) {
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
        for (int i = i0; i < i1 && ok; ++i) {
            const WorkItem it = p.work[i];
            const int L = p.seq_lens[it.b];
            const int t0 = it.t0, t1 = it.t1;
            const int nt = (t1 - t0 + kTile - 1) / kTile;
            const int ns = steps_of(t0, t1);
            const int last_vis = L - p.q_len + (row_valid ? row_seq / p.s.H : 0);
            float m_used = -CUDART_INF_F, l = 0.f;       // l: this half's share of the row sum
            bool bad_item = false;
            for (int t = 0; t < nt; ++t) bad_item |= block_of(p, it.b, t0 / kTile + t) < 0;
            for (int j = 0; j < ns && ok; ++j, ++K) {
                if (!__all_sync(0xffffffffu, mbar_wait(&bars->s_full, K & 1, bars, p.status))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (tid == 128) WTRACE(8, K);
                const int32_t nan_step = *(volatile int32_t *)&bars->nan_step;
                uint32_t sv[64];
                TMEM_LD32(lane_addr + kColS + 64 * hs, sv);
                TMEM_LD32(lane_addr + kColS + 64 * hs + 32, (sv + 32));
                tmem_wait_ld();
                const int tile_start = t0 + j * kStep + kTile * hs;
                const int n_vis = row_valid ? max(0, min(t1, last_vis + 1) - tile_start) : 0;
                // Scores stay unscaled where the scale is positive: the row max then commutes
                // with the scaling and each exponent argument is one fma. Hidden slots -> -inf.
                const bool pos_scale = p.scale_log2 > 0.f;
                const float cs = pos_scale ? p.scale_log2 : 1.f;
                if (!pos_scale || __any_sync(0xffffffffu, n_vis < kTile || nan_step == K + 1)) {
                    const volatile int32_t *at = (const volatile int32_t *)(smem + kOffNan) + kTile * hs;
#pragma unroll
                    for (int jj = 0; jj < 64; ++jj) {
                        float v = pos_scale ? __uint_as_float(sv[jj]) : __uint_as_float(sv[jj]) * p.scale_log2;
                        if (at[jj] == K + 1) v = CUDART_NAN_F;
                        sv[jj] = __float_as_uint(jj < n_vis ? v : -CUDART_INF_F);
                    }
                }
                float mx = -CUDART_INF_F;
#pragma unroll
                for (int jj = 0; jj < 64; ++jj) mx = fmaxf(mx, __uint_as_float(sv[jj]));
                mx *= cs;
                // the row's max over both halves; after it, both halves have read their S
                // columns, so P may be stored over them
                {
                    float other = -CUDART_INF_F;
                    if (!__all_sync(0xffffffffu, exchange(mx, other))) { ok = false; break; }
                    mx = fmaxf(mx, other);
                }
                if (tid == 128) WTRACE(9, K);
                float alpha = 1.f;
                bool rescale = false;
                const float m_new = fmaxf(m_used, mx);
                if (m_new > m_used + 8.f) {
                    alpha = exp2f(m_used - m_new);        // 0 when nothing was accumulated yet
                    m_used = m_new;
                    rescale = j > 0;
                }
                const float nmb = m_used == -CUDART_INF_F ? -CUDART_INF_F : -m_used;
                float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
                for (int jj = 0; jj < 32; ++jj) {
                    const float a = ex2(fmaf(__uint_as_float(sv[2 * jj]), cs, nmb));
                    const float c = ex2(fmaf(__uint_as_float(sv[2 * jj + 1]), cs, nmb));
                    const __nv_bfloat162 hh = __floats2bfloat162_rn(a, c);
                    sv[jj] = *(const uint32_t *)&hh;        // in place: scores 2 jj, 2 jj + 1 are done with
                    sum0 += a;             // fp32 row sum: the LSE does not see the rounding of P
                    sum1 += c;
                }
                l = l * alpha + (sum0 + sum1);
                // O *= alpha: the previous step's PV completed before these scores were
                // computed (the MMA thread issues a step's score MMAs after it)
                if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
                    for (int c = 4 * hs; c < 4 * hs + 4; ++c) {
                        uint32_t ov[32];
                        TMEM_LD32(lane_addr + kColO + 32 * c, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * alpha);
                        TMEM_ST32(lane_addr + kColO + 32 * c, ov);
                    }
                }
                TMEM_ST32(lane_addr + kColS + 32 * hs, sv);
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
            float l_other = 0.f;
            if (ok) ok = __all_sync(0xffffffffu, exchange(l, l_other));
            const float l_row = l + l_other;
            tc_fence_after();
            if (ok && have_next) ok = load_q_tmem();
            if (ok && have_next)
                ok = __all_sync(0xffffffffu, mbar_wait(&bars->qreg_free, (uses - 1) & 1, bars, p.status));
            const bool bad = aborted(bars) || !ok || bad_item;
            // Epilogue: O / l -> partial slot i, rounded to bf16 as the bf16 cache's (half of the
            // bytes that the combine waits for; the output is rounded as far); [32 rows x 64 dims] boxes
            // (128B-swizzled) through the region, one TMA store each; rows past the
            // sequence's rows are clipped by the tensor map.
            if (ok) {
                const float inv = l_row > 0.f ? 1.f / l_row : 0.f;
                const uint64_t keep = l2_policy_evict_last();
                uint8_t *boxes = smem + kOffQ + (warp - 4) * kEpiBoxes * kEpiBoxBytes;
                const int y = g * kRows + 32 * wq;
                const bool store = y < rows_seq;
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    const int bi = c % kEpiBoxes;
                    if (bi == 0 && c > 0) {
                        if (lane == 0) bulk_wait_read();
                        __syncwarp();
                    }
                    uint8_t *box = boxes + bi * kEpiBoxBytes;
#pragma unroll 1
                    for (int hh = 0; hh < 2; ++hh) {
                        uint32_t ov[32];
                        TMEM_LD32(lane_addr + kColO + 128 * hs + 64 * c + 32 * hh, ov);
                        tmem_wait_ld();
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
                        tma_store_3d_hint(&o_map, box, 256 * half + 128 * hs + 64 * c, y, i, keep);
                        bulk_commit();
                    }
                }
                if (lane == 0) bulk_wait_read();
                __syncwarp();
            }
            mbar_arrive(&bars->qreg_free);
            ++uses;
            if (row_valid && half == 0 && hs == 0)
                p.part_lse[(size_t)i * rows_seq + row_seq] =
                    bad || l_row != l_row ? CUDART_NAN_F : (l_row > 0.f ? m_used + log2f(l_row) : -CUDART_INF_F);
            tc_fence_before();     // O reads complete before the next item's first PV
            if (ok && have_next) ok = __all_sync(0xffffffffu, issue_q(i + 1, 1));
        }
        if (lane == 0) bulk_wait_all();   // this warp's output stores have landed
    } else if (warp >= 12) {
        // ================================================= expansion of the codes
        reg_dec<kRegsExpand>();
        // Warp e takes rows 8 e .. 8 e + 7 of a tile, four rows and a 128-byte line of each
        // (two 64-dim column blocks) at a time. Eight lanes take 16 codes each: four of one
        // row's first block and four of the neighbouring row's second, so that their 16-byte
        // stores fall on eight different swizzled chunks.
        const int e = warp - 12, p8 = lane & 7;
        const bool second = p8 >= 4;
        const int r4 = (lane >> 3) ^ (second ? 1 : 0);
        // a lane's first chunk and the shared address of its row of the warp's 8-row atom
        const uint32_t chunk = (uint32_t)((2 * (p8 & 3)) ^ r4) << 4;
        const uint32_t to0 = smem_u32(smem + kOffBuf) + (second ? kCol : 0u) + 1024u * e + 128u * r4;
        struct Rows {                      // a lane's codes of one tile, the score-only or the own dims
            uint4 c[2][2];                 // [row 4 q + r4][column block pair]
            uint2 s[2];                    // the row's eight scales of these dims
        };
        struct Step {
            int row0[2], valid[2];         // token row of each tile's first slot; its tokens
        };
        auto load = [&](Rows &x, int row0, int valid, int cb) {          // column blocks cb .. cb + 3
            const int row = 8 * e + r4;
            const size_t tok = (size_t)(row0 + row);
            const uint8_t *src = p.codes + tok * 512 + 64 * cb + 16 * p8;
            const uint8_t *scl = p.mx_scale + tok * 16 + 2 * cb;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                x.s[q] = make_uint2(0, 0);
                x.c[q][0] = x.c[q][1] = make_uint4(0, 0, 0, 0);          // zeros for slots past the end
                if (row + 4 * q < valid) {
#pragma unroll
                    for (int w = 0; w < 2; ++w)
                        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(x.c[q][w].x), "=r"(x.c[q][w].y), "=r"(x.c[q][w].z), "=r"(x.c[q][w].w)
                                     : "l"(src + 2048 * q + 128 * w));
                    asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(x.s[q].x), "=r"(x.s[q].y) : "l"(scl + 64 * q));
                }
            }
        };
        // Whether every scale is at most 1 (they take one multiplication) and every code a number.
        auto plain = [&](const Rows &x) {
            uint32_t odd = (x.s[0].x | x.s[0].y | x.s[1].x | x.s[1].y) & 0x80808080u;
#pragma unroll
            for (int q = 0; q < 2; ++q) odd |= mx_nan16(x.c[q][0]) | mx_nan16(x.c[q][1]);
            return !__any_sync(0xffffffffu, odd);
        };
        // `mark`: of own dims, the step (+ 1) to note for what is not a number; 0: of score-only
        // dims, where it is expanded to NaN; u: the tile
        auto expand = [&](const Rows &x, uint32_t to, int mark, int u, bool small) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t sw = w ? x.s[q].y : x.s[q].x;
                    uint4 o0, o1;
                    if (small) mx_expand16(x.c[q][w], mx_scale120(sw, p8 >> 1), o0, o1);
                    else {
                        uint32_t b = mx_scale_bf162((sw >> (8 * (p8 >> 1))) & 0xffu);
                        if (b == 0x7fc07fc0u || mx_nan16(x.c[q][w])) {
                            b = 0x7fc07fc0u;
                            if (mark) {
                                b = 0;
                                ((volatile int32_t *)(smem + kOffNan))[kTile * u + 8 * e + 4 * q + r4] = mark;
                                *(volatile int32_t *)&bars->nan_step = mark;
                            }
                        }
                        mx_expand16(x.c[q][w], kMx2p120, b, o0, o1);
                    }
                    // row 4 q + r4 of the warp's atom flips bit 2 of the chunk with q
                    const uint32_t at = to + 512u * q + 2u * w * kCol;
                    st_shared16(at + (chunk ^ (64u * q)), o0);
                    st_shared16(at + (chunk ^ (64u * q) ^ 16u), o1);
                }
        };
        // The steps in turn; false at the end.
        int i = i0, j = -1;
        WorkItem it = p.work[i];
        int L = p.seq_lens[it.b], nt = (it.t1 - it.t0 + kTile - 1) / kTile;
        auto next = [&](Step &st) {
            if (2 * ++j >= nt) {
                j = 0;
                if (++i >= i1) return false;
                it = p.work[i];
                L = p.seq_lens[it.b];
                nt = (it.t1 - it.t0 + kTile - 1) / kTile;
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int t = 2 * j + u;
                const int blk = t < nt ? block_of(p, it.b, it.t0 / kTile + t) : -1;
                st.row0[u] = blk * kTile;
                st.valid[u] = blk >= 0 ? min(kTile, L - (it.t0 + t * kTile)) : 0;
            }
            return true;
        };
        // Parts in turn: step K's score-only dims, its own dims, step K + 1's score-only dims
        // and so on. The loads of a part start when the part before it is expanded: the own
        // dims' have the time until the step's P . V is done to arrive, the score-only ones'
        // that until the own ones are needed again. The step after the next is looked up when
        // the next one's loads have been issued.
        Step s0, s1;                       // of K, K + 1
        Rows x, y;                         // of tile 0 and tile 1
        next(s0);
        load(x, s0.row0[0], s0.valid[0], 4 * (1 - half));
        load(y, s0.row0[1], s0.valid[1], 4 * (1 - half));
        bool more = next(s1), ok = true;
        for (int K = 0, own = 0; ok; own ^= 1) {
            const uint32_t to = to0 + 4u * (half ^ 1 ^ own) * kCol;
            // one copy of the code for both tiles
#pragma unroll 1
            for (int u = 0; u < 2; ++u) {
                // the tile's blocks are free: the score MMAs over them, or its half of P . V, are done
                uint64_t *bar = own ? &bars->empty_v[u] : &bars->empty_a;
                ok = K == 0 || (!own && u) || __all_sync(0xffffffffu, mbar_wait(bar, (K - 1) & 1, bars, p.status));
                if (!ok) break;
                WTRACE_E(own ? 14 : 12);
                expand(x, to + 8192u * u, own ? K + 1 : 0, u, plain(x));
                if (u == 0) x = y;
            }
            if (!ok) break;
            fence_proxy_async();
            mbar_arrive(own ? &bars->full_v : &bars->full_a);
            WTRACE_E(own ? 15 : 13);
            if (own) {
                if (!more) break;
                s0 = s1;
                ++K;
            }
            load(x, s0.row0[0], s0.valid[0], 4 * (half ^ own));
            load(y, s0.row0[1], s0.valid[1], 4 * (half ^ own));
            if (own) more = next(s1);
        }
        __syncwarp();
    } else {
        reg_dec<kRegsIssue>();
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
    // the register split draws on what the launch has: refuse a build that has less
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, wmx::decode_mx_kernel);
    if (e != cudaSuccess) return e;
    if (at.numRegs < wmx::kRegsLaunch) return cudaErrorInvalidConfiguration;
    dim3 grid(2, (rows_seq + wmx::kRows - 1) / wmx::kRows, p.streams);
    return launch_pdl(wmx::decode_mx_kernel, grid, dim3(wmx::kThreads), wmx::kSmemBytes, st, rope_map, q_map, o_map, p);
}

}  // namespace mla

#ifdef MLA_TRACE
extern "C" int mla_mx_trace_read(long long *events) {
    return (int)cudaMemcpyFromSymbol(events, mla::wmx::g_mxtrace, sizeof(mla::wmx::g_mxtrace));
}
#endif
