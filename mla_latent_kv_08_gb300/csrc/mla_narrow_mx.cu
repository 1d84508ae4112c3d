// Tensor-core (tcgen05 / TMEM / TMA) split-KV decode of the 8-bit latent cache for few query
// rows: at most 64 rows (draft position, head) a sequence, kv_lora_rank 512, rope 64, block
// size 64.
//
// The pair kernel (mla_wide_mx.cu) gives the query rows the MMAs' M side, 128 rows; with 64
// rows or fewer half of every product and more is padding, and both CTAs of a pair score
// every token. Here the tokens take the M side and the rows the N side, so that one CTA does
// all of a stream's work and the padding goes with N:
//
//   S^T[128 tokens x N] = K . Q^T        36 x M128 N K16, K = the step's nine column blocks
//   P^T = 2^(S^T c - m)                  a thread a token, its N rows' weights side by side
//   O^T[512 dims x N]  += V^T . P^T      4 dim tiles x 8 x M128 N K16: V^T is the same column
//                                        blocks read as an MN-major first operand, P^T an
//                                        MN-major second one
//
// The row maxima run across threads here, and any m will do that keeps the weights in the
// range of their types. So m starts at 0, and a step whose exponents all stay below 2^20
// (and, at an item's first, above 2^-20) takes one vote of the four softmax warps and no
// reduction; one that does not finds the rows' maxima and moves m there. A row that has
// seen nothing but scores of minus infinity has no maximum yet, and its first one counts as
// an item's first. Row sums stay a thread's own until the end of a work item.
//
// Measured, 64 heads over two sequences of 52k and 75k tokens: 55 us
// (the pair kernel: 64 us), bytes at the copy rate 12.4 us. The tensor pipe is busy for
// 14 % of the time: a product whose first operand lies MN-major in shared memory takes 139
// cycles, twice a K-major one, and a step's scores wait for its expansion. Taking V^T from
// a second, transposed copy would cost the room of the step after.
//
// Shared memory: nine 16 KB column blocks of a step (the rope block, done with after the
// scores, then holds P^T), Q, statistics. The blocks of dim tile c are written again for the
// next step as soon as its P . V is done, while the other tiles' run, by eight warps that
// hold a whole step's codes in registers, loaded a step ahead. (Fetching them into L2 further
// ahead as well took 3 % longer: 89.2 -> 92.3 us a call for 64 sequences of 2000 to 6000
// tokens at 32 heads.)
// Tensor memory: S^T [0,64), O^T tile c [64 + 64c, ...).
// Roles: warp 0 = Q, rope keys; warp 1 = TMEM owner, lane 0
// issues every MMA; warps 4..7 = softmax, output (thread = token, TMEM lane); warps 8..15 =
// expansion. Every wait is bounded (2 s); one that gives up records FLAG_TIMEOUT and the CTA
// winds down without trapping (the softmax warps agree on it before each barrier of theirs).
#include "mla_internal.cuh"
#include "mla_mx.cuh"
#include "mla_ptx.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>
#include <math_constants.h>
#include <string.h>

namespace mla {
namespace nmx {

using namespace ptx;

constexpr int kThreads = 512;
constexpr int kSoftThreads = 128;                     // warps 4..7
constexpr int kExpandThreads = 256;                   // warps 8..15
// Registers a thread of the four warpgroups (copies and MMA; softmax; expansion twice) once
// they are split again: what the launch had, 4 x 128.
constexpr int kRegsLaunch = 128, kRegsIssue = 80, kRegsSoft = 184, kRegsExpand = 120;
static_assert(kRegsIssue + kRegsSoft + 2 * kRegsExpand <= 4 * kRegsLaunch, "register split");
template <int N> __device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
constexpr int kTile = 64;                             // tokens per cache block
constexpr int kStep = 2 * kTile;                      // tokens per step (MMA M of the scores)
constexpr int kD = 576;                               // r + d_R
constexpr int kBlocks = 9;                            // 64-dim column blocks per token row
constexpr uint32_t kBox = kTile * 128;                // [64 tokens x 64 dims] bf16: 8 KB
constexpr uint32_t kCol = kStep * 128;                // one column block of a step: 16 KB
constexpr uint32_t kOffP = 8 * kCol;                  // P^T over the rope block
constexpr uint32_t kOffQ = kBlocks * kCol;            // 144 KB
template <int N> struct Lay {
    static constexpr uint32_t kQBlock = N * 128;      // [N rows x 64 dims] bf16
    static constexpr uint32_t kOffStat = kOffQ + kBlocks * kQBlock;   // fp32: -m [64], alpha [64], 1/l [64], per warp [4][64]
    static constexpr uint32_t kOffNan = kOffStat + 7 * 64 * 4;        // int32 [128]: 1 + the last step where the token was not a number
    static constexpr uint32_t kOffBar = kOffNan + kStep * 4;
    static constexpr uint32_t kSmemBytes = kOffBar + 256 + 1024;
    static_assert(kSmemBytes <= 232448, "shared memory budget");
};
constexpr uint32_t kColS = 0, kColO = 64;
constexpr unsigned long long kTimeoutNs = 2000000000ull;       // 2 s bounded-wait safety net
constexpr float kBound = 20.f;                        // of the exponents, log2

struct Bars {
    uint64_t full[4];         // dim tile c's two blocks are expanded
    uint64_t full_r;          // the rope block landed
    uint64_t empty[4];        // P . V over dim tile c is done
    uint64_t s_full;
    uint64_t p_full;
    uint64_t pv_done;
    uint64_t q_full, q_free;  // Q landed; the item's last scores are done
    uint64_t o_free;          // the item's output is read
    uint32_t tmem_base;
    int32_t abort_flag;
};
static_assert(sizeof(Bars) <= 256, "barriers");

// Instruction descriptor, kind::f16: bf16 A and B, fp32 accumulate, both operands MN-major.
__host__ __device__ constexpr uint32_t idesc_mn(int M, int N) { return idesc_bf16(M, N, true) | (1u << 15); }

// Shared-memory matrix descriptor: 64-byte swizzle (16-byte chunk index XOR row / 2 % 4).
__device__ __forceinline__ uint64_t sdesc64(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (sdesc(saddr, lbo, sbo) & ~((uint64_t)7 << 61)) | ((uint64_t)4 << 61);
}

__device__ __forceinline__ bool mbar_test32(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// The bounded wait for a barrier that mbar_test32 found open, out of line.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, int32_t *abort_flag, int32_t *status) {
    return mbar_wait_bounded((uint64_t *)__cvta_shared_to_generic(bar), parity, abort_flag, status, FLAG_TIMEOUT, kTimeoutNs);
}

// OR over the four softmax warps.
__device__ __forceinline__ bool soft_any(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
    return r != 0;
}
// v[0..31] (fp32 bits) of every lane, reduced over the warp: lane l gets row l's result.
template <bool MAX>
__device__ __forceinline__ float reduce_rows(uint32_t (&v)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int k = 0; k < o; ++k) {
            const uint32_t send = up ? v[k] : v[k + o], keep = up ? v[k + o] : v[k];
            const float got = __uint_as_float(__shfl_xor_sync(0xffffffffu, send, o)), own = __uint_as_float(keep);
            v[k] = __float_as_uint(MAX ? fmaxf(own, got) : own + got);
        }
    }
    return __uint_as_float(v[0]);
}

// Pipeline timestamps for performance analysis, compiled only with -DMLA_TRACE: clock64 at
// each hand-off of CTA 0 for its first kTraceSteps steps. Product builds contain none of it.
// Events: 0..3 dim tile expanded, 4 scores issued, 5 P seen, 6 P . V issued (MMA), 7 scores
// seen, 8 voted, 9 P stored (softmax), 10 tile 0 free, 11 tile 0 expanded, 12 tile 3 free,
// 13 tile 3 expanded (warp 8)
#ifdef MLA_TRACE
constexpr int kTraceSteps = 64;
__device__ long long g_nmtrace[14][kTraceSteps];
#define NTRACE(ev, step)                                                                  do {                                                                                      if (blockIdx.x == 0 && (step) < kTraceSteps) g_nmtrace[ev][step] = clock64();     } while (0)
#else
#define NTRACE(ev, step)     do {                     } while (0)
#endif

// Physical block of logical block `lb` of sequence b, or -1.
__device__ __forceinline__ int block_of(const DecodeParams &p, int b, int lb) {
    if (lb >= p.max_blocks) return -1;
    const int blk = p.block_table[(size_t)b * p.max_blocks + lb];
    return (blk >= 0 && blk < p.s.num_blocks) ? blk : -1;
}
__host__ __device__ constexpr int steps_of(int t0, int t1) { return (t1 - t0 + kStep - 1) / kStep; }

template <int N>
__global__ void __launch_bounds__(kThreads, 1)
decode_narrow_kernel(const __grid_constant__ CUtensorMap rope_map, const __grid_constant__ CUtensorMap q_map,
                     const DecodeParams p) {
    using LY = Lay<N>;
    const int stream = blockIdx.x;           // work stream (persistent over its items)
    const int rows_seq = p.q_len * p.s.H;    // at most N

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    Bars *bars = (Bars *)(smem + LY::kOffBar);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int c = 0; c < 4; ++c) {
            mbar_init(&bars->full[c], kExpandThreads);
            mbar_init(&bars->empty[c], 1);
        }
        mbar_init(&bars->full_r, 1);
        mbar_init(&bars->s_full, 1);
        mbar_init(&bars->p_full, kSoftThreads);
        mbar_init(&bars->pv_done, 1);
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->q_free, 1);
        mbar_init(&bars->o_free, kSoftThreads);
        bars->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    if (tid < kStep) ((int32_t *)(smem + LY::kOffNan))[tid] = 0;
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
    // the set-up above overlaps the planner; its schedule is read only from here on. The
    // combine may launch from here: the planner has completed, so the combine can read the
    // schedule's split ranges before its own wait.
    pdl_wait();
    pdl_trigger();
    const int i0 = p.stream_start[stream], i1 = p.stream_start[stream + 1];
    if (i0 >= i1) {                          // no work for this stream (CTA-uniform)
        if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
        return;
    }
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        return mbar_wait_bounded(bar, parity, &bars->abort_flag, p.status, FLAG_TIMEOUT, kTimeoutNs);
    };

    if (warp == 0) {
        // ================================================= Q, rope keys
        reg_dec<kRegsIssue>();
        if (lane == 0) {
            const int oob_row = p.s.num_blocks * kTile;       // past the end: TMA fills zeros
            int K = 0, items = 0;
            bool ok = true;
            for (int i = i0; i < i1 && ok; ++i) {
                const WorkItem it = p.work[i];
                const int nt = (it.t1 - it.t0 + kTile - 1) / kTile, ns = steps_of(it.t0, it.t1);
                if (items > 0 && !wait(&bars->q_free, (items - 1) & 1)) break;
                mbar_expect_tx(&bars->q_full, kBlocks * LY::kQBlock);
                // rows behind the sequence's last belong to the next one; their columns are not stored
                for (int c = 0; c < kBlocks; ++c)
                    tma_load_2d(smem + kOffQ + c * LY::kQBlock, &q_map, 64 * c, it.b * rows_seq, &bars->q_full);
                ++items;
                for (int j = 0; j < ns; ++j, ++K) {
                    // a missing or bad block reads zeros past the end (the softmax marks a bad
                    // block's rows NaN)
                    int row0[2];
                    for (int u = 0; u < 2; ++u) {
                        const int blk = 2 * j + u < nt ? block_of(p, it.b, it.t0 / kTile + 2 * j + u) : -1;
                        if (2 * j + u < nt && blk < 0) raise_flag(p.status, FLAG_BAD_BLOCK);
                        row0[u] = blk >= 0 ? blk * kTile : oob_row;
                    }
                    // the rope block holds the last step's P^T until its P . V is done
                    if (K > 0 && !wait(&bars->pv_done, (K - 1) & 1)) { ok = false; break; }
                    mbar_expect_tx(&bars->full_r, 2 * kBox);
                    tma_load_2d(smem + kOffP, &rope_map, 0, row0[0], &bars->full_r);
                    tma_load_2d(smem + kOffP + kBox, &rope_map, 0, row0[1], &bars->full_r);
                }
            }
            // never leave a copy in flight into this CTA's shared memory
            if (items > 0) mbar_drain(&bars->q_full, (items - 1) & 1);
            if (K > 0) mbar_drain(&bars->full_r, (K - 1) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================================================= MMA issuer: lane 0 alone
        reg_dec<kRegsIssue>();
        if (lane == 0) {
            constexpr uint32_t kIdS = idesc_bf16(128, N, false), kIdO = idesc_mn(128, N);
            const uint64_t kd = sdesc(smem_u32(smem), 16, 1024);
            const uint64_t qd = sdesc(smem_u32(smem + kOffQ), 16, 1024);
            // MN-major: 64-dim atoms a column block apart, 8-token groups 1 KB apart
            const uint64_t vd = sdesc(smem_u32(smem), kCol, 1024);
            // P^T: rows of 128 bytes in the 128-byte swizzle, or (N = 32) of 64 in the 64-byte one
            const uint64_t pd = N > 32 ? sdesc(smem_u32(smem + kOffP), kCol, 1024) : sdesc64(smem_u32(smem + kOffP), kCol, 512);
            constexpr uint32_t kPStep = N > 32 ? 128 : 64;     // 16 tokens, in 16-byte units
            const uint32_t d_s = tmem + kColS;
            // The thread's own pace counts here (68 products of few columns a step): the first
            // probe of a barrier is inline, the bounded wait out of line.
            const uint32_t full0 = smem_u32(&bars->full[0]), full_r = smem_u32(&bars->full_r), p_full = smem_u32(&bars->p_full);
            auto there = [&](uint32_t bar, uint32_t parity) {
                return mbar_test32(bar, parity) || wait_slow(bar, parity, &bars->abort_flag, p.status);
            };
            bool ok = true;
            int K = 0, items = 0;
            for (int i = i0; i < i1 && ok; ++i, ++items) {
                const WorkItem it = p.work[i];
                const int ns = steps_of(it.t0, it.t1);
                ok = wait(&bars->q_full, items & 1);
                for (int j = 0; j < ns && ok; ++j, ++K) {
                    // scores, a dim tile's two blocks as they are expanded (descriptor start
                    // addresses advance in 16-byte units)
                    uint64_t a = kd, b = qd;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        ok = there(full0 + 8 * c, K & 1);
                        if (!ok) break;
                        NTRACE(c, K);
                        tc_fence_after();
                        mma_ss(d_s, a, b, kIdS, c > 0 ? 1u : 0u);
#pragma unroll
                        for (int e = 1; e < 8; ++e)
                            mma_ss_k<kIdS, 1>(d_s, a + (uint64_t)(((e >> 2) * kCol + 32 * (e & 3)) >> 4),
                                              b + (uint64_t)(((e >> 2) * LY::kQBlock + 32 * (e & 3)) >> 4));
                        a += (2 * kCol) >> 4;
                        b += (2 * LY::kQBlock) >> 4;
                    }
                    ok = ok && there(full_r, K & 1);
                    if (!ok) break;
#pragma unroll
                    for (int e = 0; e < 4; ++e) mma_ss_k<kIdS, 1>(d_s, a + 2 * e, b + 2 * e);
                    mma_commit(&bars->s_full);
                    NTRACE(4, K);
                    if (j + 1 == ns) mma_commit(&bars->q_free);
                    // P . V, a dim tile at a time: its blocks are free as soon as it is done
                    if (j == 0 && items > 0) ok = wait(&bars->o_free, (items - 1) & 1);
                    ok = ok && there(p_full, K & 1);
                    if (!ok) break;
                    NTRACE(5, K);
                    tc_fence_after();
                    uint64_t v = vd;
                    uint32_t d_o = tmem + kColO;
                    uint64_t *bar = &bars->empty[0];
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        mma_ss(d_o, v, pd, kIdO, j > 0 ? 1u : 0u);
#pragma unroll
                        for (int e = 1; e < 8; ++e) mma_ss_k<kIdO, 1>(d_o, v + 128 * e, pd + kPStep * e);
                        mma_commit(bar++);
                        v += (2 * kCol) >> 4;
                        d_o += 64;
                    }
                    mma_commit(&bars->pv_done);
                    NTRACE(6, K);
                }
            }
            // products in flight must end before the tensor memory is given back
            if (!ok) mma_commit(&bars->pv_done);
            if (K > 0 || !ok) mbar_drain(&bars->pv_done, (ok ? K - 1 : K) & 1);
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        // ================================================= softmax and output
        reg_inc<kRegsSoft>();
        const int wq = warp & 3, tok_row = 32 * wq + lane;     // this thread's token of a step
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * wq) << 16);
        const uint32_t p_row = smem_u32(smem + kOffP) + (N > 32 ? 128u : 64u) * tok_row;
        const uint32_t p_swz = N > 32 ? tok_row & 7 : (tok_row >> 1) & 3;
        float *nm_s = (float *)(smem + LY::kOffStat), *alpha_s = nm_s + 64, *inv_s = nm_s + 128, *red_s = nm_s + 192;
        const float c2 = p.scale_log2;
        bool ok = true;
        int K = 0;
        for (int i = i0; i < i1 && ok; ++i) {
            const WorkItem it = p.work[i];
            const int L = p.seq_lens[it.b];
            const int nt = (it.t1 - it.t0 + kTile - 1) / kTile, ns = steps_of(it.t0, it.t1);
            bool bad_item = false;
            for (int t = 0; t < nt; ++t) bad_item |= block_of(p, it.b, it.t0 / kTile + t) < 0;
            float l[N];                                        // this thread's share of the row sums
#pragma unroll
            for (int n = 0; n < N; ++n) l[n] = 0.f;
            if (tok_row < 64) nm_s[tok_row] = 0.f;             // m = 0 until the first scores
            // whether row tok_row has its m (a row that does not see the item's first token sees
            // none of it and needs none), and whether a row is still without
            bool set = tok_row >= N || tok_row < max(0, it.t0 - (L - p.q_len)) * p.s.H, first = true;
            soft_any(false);
            for (int j = 0; j < ns; ++j, ++K) {
                const bool mine_ok = __all_sync(0xffffffffu, wait(&bars->s_full, K & 1));
                tc_fence_after();
                if (tok_row == 0) NTRACE(7, K);
                const int tok = it.t0 + j * kStep + tok_row;
                // rows before n_min do not see this token (drafts; or the slot is past the end)
                // (clamped before the product: at most q_len * H, where a long cache's tokens times
                // heads pass 2^31)
                const int n_min = tok >= it.t1 ? N : max(0, tok - (L - p.q_len)) * p.s.H;
                const bool not_a_number = ((volatile int32_t *)(smem + LY::kOffNan))[tok_row] == K + 1;
                // exponents of 32 rows, over the rows' m; hidden ones -inf
                uint32_t sv[32];
                auto exponents = [&](int h) {
                    TMEM_LD32(lane_addr + kColS + 32 * h, sv);
                    tmem_wait_ld(sv);
#pragma unroll
                    for (int n4 = 0; n4 < 32; n4 += 4) {
                        const float4 nm = *(const float4 *)(nm_s + 32 * h + n4);
                        sv[n4] = __float_as_uint(fmaf(__uint_as_float(sv[n4]), c2, nm.x));
                        sv[n4 + 1] = __float_as_uint(fmaf(__uint_as_float(sv[n4 + 1]), c2, nm.y));
                        sv[n4 + 2] = __float_as_uint(fmaf(__uint_as_float(sv[n4 + 2]), c2, nm.z));
                        sv[n4 + 3] = __float_as_uint(fmaf(__uint_as_float(sv[n4 + 3]), c2, nm.w));
                    }
                    if (__any_sync(0xffffffffu, n_min > 32 * h)) {
#pragma unroll
                        for (int n = 0; n < 32; ++n)
                            if (32 * h + n < n_min) sv[n] = __float_as_uint(-CUDART_INF_F);
                    }
                    if (not_a_number) {
#pragma unroll
                        for (int n = 0; n < 32; ++n)
                            if (32 * h + n >= n_min) sv[n] = 0x7fc00000u;
                    }
                };
                float top = -CUDART_INF_F, low = CUDART_INF_F; // the largest and the least visible exponent
#pragma unroll 1
                for (int h = 0; h < N / 32; ++h) {
                    exponents(h);
#pragma unroll
                    for (int n = 0; n < 32; ++n) top = fmaxf(top, __uint_as_float(sv[n]));
                    if (first)
#pragma unroll
                        for (int n = 0; n < 32; ++n) low = fminf(low, 32 * h + n < n_min ? 0.f : __uint_as_float(sv[n]));
                }
                const bool slow = soft_any(top > kBound || (first && low < -kBound) || !mine_ok);
                if (tok_row == 0) NTRACE(8, K);
                if (slow) {
                    ok = !soft_any(!mine_ok);
                    if (!ok) break;
                    // The maxima of every row over the step's tokens; m becomes them where the row
                    // has none yet, and rises to them later where they are past the bound.
#pragma unroll 1
                    for (int h = 0; h < N / 32; ++h) {
                        exponents(h);
                        red_s[64 * wq + 32 * h + lane] = reduce_rows<true>(sv);
                    }
                    soft_any(false);
                    if (tok_row < N) {
                        const float d = fmaxf(fmaxf(red_s[tok_row], red_s[64 + tok_row]),
                                              fmaxf(red_s[128 + tok_row], red_s[192 + tok_row]));
                        const bool raise = d != -CUDART_INF_F && (!set || d > kBound);
                        alpha_s[tok_row] = raise && set ? exp2f(-d) : 1.f;
                        if (raise) {
                            nm_s[tok_row] -= d;
                            set = true;
                        }
                    }
                    first = soft_any(!set);
#pragma unroll
                    for (int n = 0; n < N; ++n) l[n] *= alpha_s[n];
                    // O^T *= alpha: the scores' barrier says that the P . V before is done
                    if (j > 0) {
#pragma unroll 1
                        for (int c = 0; c < 4 * (N / 32); ++c) {
                            const uint32_t at = lane_addr + kColO + 64 * (c / (N / 32)) + 32 * (c % (N / 32));
                            TMEM_LD32(at, sv);
                            tmem_wait_ld(sv);
                            const float *al = alpha_s + 32 * (c % (N / 32));
#pragma unroll
                            for (int n = 0; n < 32; ++n) sv[n] = __float_as_uint(__uint_as_float(sv[n]) * al[n]);
                            TMEM_ST32(at, sv);
                        }
                        tmem_wait_st();
                    }
                } else {
                    set = true;
                    first = false;
                }
                // weights (bf16) into the token's row of P^T, 16-byte chunks swizzled as an
                // MN-major operand; sums of the unrounded ones
#pragma unroll
                for (int h = 0; h < N / 32; ++h) {
                    if (N > 32 || slow) exponents(h);          // (else they are still there)
#pragma unroll
                    for (int ch = 0; ch < 4; ++ch) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = ex2(__uint_as_float(sv[8 * ch + 2 * e])), y = ex2(__uint_as_float(sv[8 * ch + 2 * e + 1]));
                            l[32 * h + 8 * ch + 2 * e] += x;
                            l[32 * h + 8 * ch + 2 * e + 1] += y;
                            const __nv_bfloat162 h2 = __floats2bfloat162_rn(x, y);
                            w[e] = *(const uint32_t *)&h2;
                        }
                        st_shared16(p_row + (((uint32_t)(4 * h + ch) ^ p_swz) << 4), make_uint4(w[0], w[1], w[2], w[3]));
                    }
                }
                tc_fence_before();
                fence_proxy_async();
                mbar_arrive(&bars->p_full);
                if (tok_row == 0) NTRACE(9, K);
            }
            if (!ok) break;
            ok = __all_sync(0xffffffffu, wait(&bars->pv_done, (K - 1) & 1));
            ok = !soft_any(!ok);
            if (!ok) break;
            tc_fence_after();
            // row sums over the tokens, then O^T / l into the item's partial slot, rounded to bf16
            // as the pair kernel's (half of the bytes that the combine waits for)
#pragma unroll
            for (int h = 0; h < N / 32; ++h) {
                uint32_t v[32];
#pragma unroll
                for (int n = 0; n < 32; ++n) v[n] = __float_as_uint(l[32 * h + n]);
                red_s[64 * wq + 32 * h + lane] = reduce_rows<false>(v);
            }
            soft_any(false);
            if (tok_row < N) {
                const float s = (red_s[tok_row] + red_s[64 + tok_row]) + (red_s[128 + tok_row] + red_s[192 + tok_row]);
                inv_s[tok_row] = s > 0.f ? 1.f / s : 0.f;
                if (tok_row < rows_seq)
                    p.part_lse[(size_t)i * rows_seq + tok_row] =
                        bad_item || s != s ? CUDART_NAN_F : (s > 0.f ? log2f(s) - nm_s[tok_row] : -CUDART_INF_F);
            }
            soft_any(false);
            __nv_bfloat16 *part = (__nv_bfloat16 *)p.part_o + (size_t)i * rows_seq * 512;
#pragma unroll 1
            for (int c = 0; c < 4 * (N / 32); ++c) {
                const int tile = c / (N / 32), n0 = 32 * (c % (N / 32));
                uint32_t ov[32];
                TMEM_LD32(lane_addr + kColO + 64 * tile + n0, ov);
                tmem_wait_ld(ov);
                // two lanes' dims side by side: the even lane stores row n, the odd one row n + 1
                __nv_bfloat16 *dst = part + 128 * tile + 32 * wq + (lane & ~1);
#pragma unroll
                for (int n = 0; n < 32; n += 2) {
                    const float x = __uint_as_float(ov[n]) * inv_s[n0 + n], y = __uint_as_float(ov[n + 1]) * inv_s[n0 + n + 1];
                    const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? x : y, 1);
                    const __nv_bfloat162 h2 = lane & 1 ? __floats2bfloat162_rn(got, y) : __floats2bfloat162_rn(x, got);
                    const int row = n0 + n + (lane & 1);
                    if (row < rows_seq) *(__nv_bfloat162 *)(dst + (size_t)row * 512) = h2;
                }
            }
            tc_fence_before();
            mbar_arrive(&bars->o_free);
        }
        __syncwarp();
    } else if (warp >= 8) {
        // ================================================= expansion of the codes
        // Warp e takes rows 16 e .. 16 e + 15 of the step, four rows and a 128-byte line of each
        // (a dim tile's two column blocks) at a time. Eight lanes take 16 codes each: four of
        // one row's first block and four of the neighbouring row's second, so that their
        // 16-byte stores fall on eight different swizzled chunks.
        reg_dec<kRegsExpand>();
        const int e = warp - 8, p8 = lane & 7;
        const bool second = p8 >= 4;
        const int r4 = (lane >> 3) ^ (second ? 1 : 0);
        const uint32_t chunk = (uint32_t)((2 * (p8 & 3)) ^ r4) << 4;
        const uint32_t to0 = smem_u32(smem) + (second ? kCol : 0u) + 2048u * e + 128u * r4;
        struct Rows {                      // a lane's codes of one dim tile
            uint4 c[4];                    // row 4 q + r4
            uint32_t s[4];                 // the row's four scales of these dims
        };
        struct Half {                      // the tile of the step that the warp's rows are in
            int row0, valid;
        };
        auto load = [&](Rows &x, const Half &st, int c) {
            const int row = 16 * (e & 3) + r4;
            const size_t tok = (size_t)(st.row0 + row);
            const uint8_t *src = p.codes + tok * 512 + 128 * c + 16 * p8;
            const uint8_t *scl = p.mx_scale + tok * 16 + 4 * c;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                x.s[q] = 0;
                x.c[q] = make_uint4(0, 0, 0, 0);               // zeros for slots past the end
                if (row + 4 * q < st.valid) {
                    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(x.c[q].x), "=r"(x.c[q].y), "=r"(x.c[q].z), "=r"(x.c[q].w)
                                 : "l"(src + 2048 * q));
                    asm volatile("ld.global.u32 %0, [%1];" : "=r"(x.s[q]) : "l"(scl + 64 * q));
                }
            }
        };
        // Whether every scale is at most 1 (they take one multiplication) and every code a number.
        auto plain = [&](const Rows &x) {
            uint32_t odd = (x.s[0] | x.s[1] | x.s[2] | x.s[3]) & 0x80808080u;
#pragma unroll
            for (int q = 0; q < 4; ++q) odd |= mx_nan16(x.c[q]);
            return !__any_sync(0xffffffffu, odd);
        };
        // A group that is not a number, or a lane's codes with one that is not, become zeros
        // (their product with a hidden row's weight 0 stays 0) and their token is noted with
        // `mark`, so that the scores of the rows that see it become NaN.
        auto expand = [&](const Rows &x, uint32_t to, int mark, bool small) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint4 o0, o1;
                if (small) mx_expand16(x.c[q], mx_scale120(x.s[q], p8 >> 1), o0, o1);
                else {
                    uint32_t b = mx_scale_bf162((x.s[q] >> (8 * (p8 >> 1))) & 0xffu);
                    if (b == 0x7fc07fc0u || mx_nan16(x.c[q])) {
                        b = 0;
                        ((volatile int32_t *)(smem + LY::kOffNan))[16 * e + 4 * q + r4] = mark;
                    }
                    mx_expand16(x.c[q], kMx2p120, b, o0, o1);
                }
                // row 4 q + r4 of the warp's two atoms flips bit 2 of the chunk with q
                st_shared16(to + 512u * q + (chunk ^ (64u * (q & 1))), o0);
                st_shared16(to + 512u * q + (chunk ^ (64u * (q & 1)) ^ 16u), o1);
            }
        };
        int i = i0, j = -1;
        WorkItem it = p.work[i];
        int L = p.seq_lens[it.b], nt = (it.t1 - it.t0 + kTile - 1) / kTile;
        auto next = [&](Half &st) {                            // the steps in turn; false at the end
            if (2 * ++j >= nt) {
                j = 0;
                if (++i >= i1) return false;
                it = p.work[i];
                L = p.seq_lens[it.b];
                nt = (it.t1 - it.t0 + kTile - 1) / kTile;
            }
            const int t = 2 * j + (e >> 2);
            const int blk = t < nt ? block_of(p, it.b, it.t0 / kTile + t) : -1;
            st.row0 = blk * kTile;
            st.valid = blk >= 0 ? min(kTile, L - (it.t0 + t * kTile)) : 0;
            return true;
        };
        Half s0;
        Rows x0, x1, x2, x3;               // the step's dim tiles
        next(s0);
        load(x0, s0, 0);
        load(x1, s0, 1);
        load(x2, s0, 2);
        load(x3, s0, 3);
        bool more = next(s0);
        for (int K = 0;; ++K) {
            auto part = [&](Rows &x, int c) {
                if (K > 0 && !__all_sync(0xffffffffu, wait(&bars->empty[c], (K - 1) & 1))) return false;
                if (tid == 256 && c % 3 == 0) NTRACE(c == 0 ? 10 : 12, K);
                expand(x, to0 + 2u * c * kCol, K + 1, plain(x));
                fence_proxy_async();
                mbar_arrive(&bars->full[c]);
                if (tid == 256 && c % 3 == 0) NTRACE(c == 0 ? 11 : 13, K);
                return true;
            };
            if (!part(x0, 0) || !part(x1, 1) || !part(x2, 2) || !part(x3, 3) || !more) break;
            // all the next step's loads at once, after the last use of this one's (loads share
            // the few counters that a use waits for)
            load(x0, s0, 0);
            load(x1, s0, 1);
            load(x2, s0, 2);
            load(x3, s0, 3);
            more = next(s0);
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

template <int N>
static cudaError_t launch(const DecodeParams &p, cudaStream_t st) {
    CUtensorMap rope_map, q_map;
    if (!make_map(&rope_map, p.rope, (uint64_t)p.s.num_blocks * p.s.bs, kTile, (uint64_t)p.s.dR) ||
        !make_map(&q_map, p.q, (uint64_t)p.B * p.q_len * p.s.H, N, kD))
        return cudaErrorInvalidValue;
    auto kern = decode_narrow_kernel<N>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Lay<N>::kSmemBytes);
    if (e != cudaSuccess) return e;
    // the register split draws on what the launch has: refuse a build that has less
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, kern);
    if (e != cudaSuccess) return e;
    if (at.numRegs < kRegsLaunch) return cudaErrorInvalidConfiguration;
    return launch_pdl(kern, dim3(p.streams), dim3(kThreads), Lay<N>::kSmemBytes, st, rope_map, q_map, p);
}

}  // namespace nmx

bool decode_narrow_supported(const ShapeArgs &s, int32_t q_len) { return is_mx(s.kind) && (long long)q_len * s.H <= 64; }

// A step of this kernel takes 1.26 (32 columns) to 1.5 (64) times the pair kernel's, on one
// SM instead of two, but its first step costs more. Measured calls, pair / this, at 16 rows:
// 26.8 / 26.0 us for 32 sequences of 300 tokens, 39.5 / 32.6 of 1250, 87.0 / 62.2 of 5000;
// one sequence of 169 tokens 18.2 / 20.4. At 64 rows: 28.0 / 33.5 us of 600, 39.5 / 39.9 of
// 1250, 55.1 / 51.0 of 2500, 85.5 / 72.1 of 5000. So: from one step a CTA on for 32 columns,
// from four on for 64. The tokens are what the block table has room for (the lengths are on
// the device); the figures are of tables as wide as the longest sequence. Under a wider one, as
// a server has for its longest context, the rule takes this kernel for shorter sequences too,
// at the cost that the figures show (5.5 us of 28 for those of 600 tokens), and the same
// sequences may then round differently.
bool decode_narrow_wins(const ShapeArgs &s, int32_t q_len, int64_t tokens, int32_t sms) {
    return tokens >= (int64_t)(q_len * s.H <= 32 ? 1 : 4) * nmx::kStep * sms;
}

cudaError_t launch_decode_narrow(const DecodeParams &p, cudaStream_t st) {
    return p.q_len * p.s.H <= 32 ? nmx::launch<32>(p, st) : nmx::launch<64>(p, st);
}

}  // namespace mla

#ifdef MLA_TRACE
extern "C" int mla_narrow_trace_read(long long *events) {
    return (int)cudaMemcpyFromSymbol(events, mla::nmx::g_nmtrace, sizeof(mla::nmx::g_nmtrace));
}
#endif
