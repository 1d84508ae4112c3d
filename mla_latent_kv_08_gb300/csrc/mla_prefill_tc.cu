// Prefill on the tensor cores (tcgen05 / TMEM / TMA) for the DeepSeek-V3 latent:
// kv_lora_rank 512, rope 64, nope 128, v_head_dim 128, bf16 rows (BF16 and MXFP8 caches).
//
// expand_tc_kernel    K[h] = rows . W_UK[h]^T and V[h] = rows . W_UV[h] for the heads of
//                     a pass, bf16 out
// prefill_tc_kernel   causal attention of 256 new tokens of one head over K, V and the
//                     rope keys in the dense rows
//
// Every wait is bounded (2 s): one that gives up records FLAG_TIMEOUT and the CTA winds
// down without trapping. The attention's own rows become NaN then; after one of the
// expansion's, whose keys and values are what was in the workspace, all rows do.
#include "mla_internal.cuh"
#include "mla_ptx.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>
#include <limits.h>
#include <math_constants.h>
#include <string.h>

namespace mla {
namespace pf {

using namespace ptx;

constexpr unsigned long long kTimeoutNs = 2000000000ull;       // 2 s bounded-wait safety net
constexpr int kR = 512, kRope = 64, kDn = 128, kDv = 128;
constexpr uint32_t kBlock = 128 * 128;                // [128 rows x 64 values] bf16: 16 KB

// ---- the pair: copies that report to CTA 0, products over both SMs ----------
__device__ __forceinline__ void tma_pair_2d(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_u32(dst)), "l"((uint64_t)map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_pair_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(smem_u32(dst)), "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void mma2_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
template <uint32_t IDESC, int ACC>
__device__ __forceinline__ void mma2_ss(uint32_t d_tmem, uint64_t a, uint64_t b) {
    asm volatile("tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, %4;" ::"r"(d_tmem), "l"(a), "l"(b), "n"(IDESC), "n"(ACC)
                 : "memory");
}
__device__ __forceinline__ void mma2_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void prefetch_2d(const CUtensorMap *map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"((uint64_t)map), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void prefetch_3d(const CUtensorMap *map, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"((uint64_t)map), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
// Arrives, once the products issued so far are done, on this barrier of both CTAs.
__device__ __forceinline__ void commit2(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_u32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
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
// An arrival on a barrier of either CTA of the pair. What it reports is in tensor memory,
// complete (tcgen05.wait::st) and ordered by the tcgen05 fences on both sides; no other
// memory hangs on it, so it needs no cluster-wide release (which took a thousand cycles and
// more: it waits for every access of the thread).
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
template <int N> __device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// ============================================================================
// Keys and values. A pair of CTAs makes 256 rows of two heads' keys, then of their values, then
// the next two heads: the rows' 512 latent dims stay in shared memory (CTA r holds rows 128 r
// .. 128 r + 127, 128 KB), only weights stream through it, CTA r holding head r's of the two.
// So a CTA reads 128 KB of L2 per head for 67 MFLOP, 32 bytes a cycle at full rate; a tile of
// its own of 256 x 256 reads twice that. Each product is M256 N256 K16 (the two heads'
// columns). Keys and values have accumulators of their own, the whole of tensor memory, so
// that one is rounded and stored while the other is made. W_UK[h] is K-major as it lies
// ([d_n, r]), W_UV[h] MN-major ([r, d_v]).
//
// They are rounded to bf16, the type of the next products' operands. Measured: 37k rows on
// 128 heads 0.78 ms, 1.57 PFLOP/s (cuBLAS in a loop of seconds 1.74); 28k rows on 16 heads
// 89 us. Without pairs 1.21 ms. Bound by the tensor pipe and, on long ones, the power cap.
// ============================================================================
namespace ex {
constexpr int kThreads = 384;                          // warp 0 copies, 1 products (CTA 0), 4..11 output
constexpr int kStages = 5;
constexpr uint32_t kStage = kBlock;                    // 64 dims of a head's 128 columns: 16 KB
constexpr int kChunks = kR / 64;
constexpr uint32_t kOffW = kChunks * kBlock;           // after the rows
constexpr uint32_t kOffOut = kOffW + kStages * kStage; // a 2 KB box a warp: 32 rows x 32 columns
constexpr uint32_t kOffBar = kOffOut + 8 * 2048;
constexpr uint32_t kSmemBytes = kOffBar + 256 + 1024;  // + alignment slack
static_assert(kSmemBytes <= 232448, "shared memory budget");

struct Bars {
    // of CTA 0: both CTAs' rows and weights landed; both CTAs' outputs of an accumulator are read
    uint64_t rows_full, full[kStages], acc_free[2];
    // of each CTA, from CTA 0's products
    uint64_t empty[kStages], acc_full[2];
    uint32_t tmem_base;
    int32_t abort_flag;
};
static_assert(sizeof(Bars) <= 256, "barriers");

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
expand_tc_kernel(const __grid_constant__ CUtensorMap rows_map, const __grid_constant__ CUtensorMap uk_map,
                 const __grid_constant__ CUtensorMap uv_map, const PrefillParams p, int heads) {
    const int r = (int)cluster_ctarank(), m0 = (blockIdx.x >> 1) * 256;
    pdl_trigger();
    pdl_wait();
    const int rows_used = p.kv_off[p.B];
    if (m0 >= rows_used) return;                       // both CTAs of a pair
    const int hl0 = blockIdx.y * heads, nh = min(heads, p.nh - hl0);     // heads of this pass (`heads` is even)
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    Bars *bars = (Bars *)(smem + kOffBar);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        mbar_init(&bars->rows_full, 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars->acc_full[s], 1);
            mbar_init(&bars->acc_free[s], 16);         // a warp of either CTA an arrival
        }
        bars->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&bars->tmem_base)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();                        // the other CTA's barriers and tensor memory are there
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        return mbar_wait_bounded(bar, parity, &bars->abort_flag, p.status, FLAG_TIMEOUT, kTimeoutNs);
    };
    const int parts = 2 * ((nh + 1) / 2), turns = parts * kChunks;       // a part: two heads' keys or values
    if (warp == 0) {
        if (lane == 0) {
            auto leader = [&](uint64_t *bar) { return mapa(smem_u32(bar), 0); };
            if (r == 0) mbar_expect_tx(&bars->rows_full, 2 * kChunks * kBlock);
            for (int c = 0; c < kChunks; ++c)          // rows past the end read zeros
                tma_pair_2d(smem + c * kBlock, &rows_map, 64 * c, m0 + 128 * r, leader(&bars->rows_full));
            int u = 0;
            for (; u < turns; ++u) {
                const int s = u % kStages, use = u / kStages, c = u % kChunks, part = u / kChunks;
                // this CTA's head; behind the pass's last one its products are not stored (and
                // behind the layer's last one it reads zeros)
                const int h = p.h0 + hl0 + 2 * (part >> 1) + r;
                if (use > 0 && !wait(&bars->empty[s], (use - 1) & 1)) break;
                if (r == 0) mbar_expect_tx(&bars->full[s], 2 * kStage);
                uint8_t *st = smem + kOffW + s * kStage;
                const uint32_t bar = leader(&bars->full[s]);
                if ((part & 1) == 0) {
                    tma_pair_2d(st, &uk_map, 64 * c, h * kDn, bar);
                } else {
                    tma_pair_2d(st, &uv_map, 0, h * kR + 64 * c, bar);
                    tma_pair_2d(st + kBlock / 2, &uv_map, 64, h * kR + 64 * c, bar);
                }
            }
            // Never leave a copy in flight into the pair's shared memory: CTA 0 waits here for
            // both CTAs' copies, CTA 1 for CTA 0 at the end.
            if (r == 0) {
                mbar_drain(&bars->rows_full, 0);
                for (int v = max(0, u - kStages); v < u; ++v) mbar_drain(&bars->full[v % kStages], (v / kStages) & 1);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && r == 0) {
            constexpr uint32_t kIdK = idesc_bf16(256, 256, false), kIdV = idesc_bf16(256, 256, true);
            const uint64_t rows = sdesc(smem_u32(smem), 16, 1024);
            const uint64_t wk = sdesc(smem_u32(smem + kOffW), 16, 1024);
            const uint64_t wv = sdesc(smem_u32(smem + kOffW), kBlock / 2, 1024);         // MN-major
            const uint32_t full0 = smem_u32(&bars->full[0]), free0 = smem_u32(&bars->acc_free[0]);
            auto there = [&](uint32_t bar, uint32_t parity) {
                return mbar_test32(bar, parity) || wait_slow(bar, parity, &bars->abort_flag, p.status);
            };
            bool ok = wait(&bars->rows_full, 0);
            int s = 0;
            uint32_t ph = 0;                           // stage, phase of its use
            for (int i = 0; i < parts && ok; ++i) {
                const int v = i & 1;                   // keys, values
                const uint32_t d = tmem + 256 * v, idesc = v ? kIdV : kIdK, step = v ? 128 : 2;
                ok = i < 2 || there(free0 + 8 * v, ((i >> 1) - 1) & 1);
                uint64_t a = rows;
#pragma unroll 1
                for (int c = 0; c < kChunks && ok; ++c) {
                    ok = there(full0 + 8 * s, ph);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t w = (v ? wv : wk) + (uint64_t)(s * (kStage >> 4));
#pragma unroll
                    for (int e = 0; e < 4; ++e) mma2_ss(d, a + 2 * e, w + step * e, idesc, (c > 0 || e > 0) ? 1u : 0u);
                    commit2(&bars->empty[s]);
                    a += kBlock >> 4;
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
                commit2(&bars->acc_full[v]);
            }
            // products in flight must end before the tensor memory is given back
            mbar_drain(&bars->acc_full[1], ((parts >> 1) - 1) & 1);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // warp w: rows 32*(w%4)..+31 (its tensor-memory lanes) of the first (w < 8) or second head
        const int q = warp & 3, hv = (warp - 4) >> 2;
        const int row = m0 + 128 * r + 32 * q;
        uint8_t *box = smem + kOffOut + (warp - 4) * 2048;
        // A latent with a NaN or an infinity: NaN keys, so that every new token that sees it is
        // NaN, and zero values, so that those whose mask hides it (weight 0) do not.
        const bool odd = row < rows_used && p.odd[row + lane], any_odd = __any_sync(0xffffffffu, odd);
        for (int i = 0; i < parts; ++i) {
            const int v = i & 1, hl = hl0 + (i & ~1) + hv;
            if (!__all_sync(0xffffffffu, wait(&bars->acc_full[v], (i >> 1) & 1))) break;
            tc_fence_after();
            const uint32_t at = tmem + ((uint32_t)(32 * q) << 16) + 256 * v + 128 * hv;
            const bool store = row < rows_used && hl < hl0 + nh;
            // a lane's place of the stores: row lane / 4 of eight, 16 bytes lane % 4
            __nv_bfloat16 *dst = (__nv_bfloat16 *)(v ? p.v : p.k) + ((size_t)hl * p.cap_rows + row + (lane >> 2)) * 128 + 8 * (lane & 3);
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {              // 32 columns
                uint32_t x[32];
                TMEM_LD32(at + 32 * c, x);
                tmem_wait_ld();
                if (c == 3) {                          // the accumulator is read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_cluster(mapa(smem_u32(&bars->acc_free[v]), 0));
                }
                if (any_odd) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = odd ? (v ? 0u : 0x7fc00000u) : x[e];
                }
                // rows of 64 bytes, 16-byte chunks rotated by the row pair
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(x[8 * ch + 2 * e]),
                                                                       __uint_as_float(x[8 * ch + 2 * e + 1]));
                        w[e] = *(const uint32_t *)&y;
                    }
                    *(uint4 *)(box + lane * 64 + ((ch ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                __syncwarp();
                if (store) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {      // rows 8 g + lane / 4
                        const int rr = 8 * g + (lane >> 2);
                        *(uint4 *)(dst + (size_t)(8 * g) * 128 + 32 * c) =
                            *(const uint4 *)(box + rr * 64 + (((lane & 3) ^ ((rr >> 1) & 3)) << 4));
                    }
                }
                __syncwarp();
            }
        }
    }
    // neither CTA leaves while the other may reach its barriers, its shared memory or its
    // tensor memory
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (tid == 0 && bars->abort_flag) p.status[1] = 1;
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}
}  // namespace ex

// ============================================================================
// Attention. A pair of CTAs (a cluster of two) takes 256 new tokens of one sequence for one
// head, 128 rows a CTA, over 128-token steps of the cache:
//
//   S[256 x 128] = Q . K^T   12 x M256 N128 K16 over both SMs
//   P = 2^(S c - m)          a thread a row: no shuffles
//   O[256 x 128] += P . V    8 x M256 N128 K16, P from tensor memory
//
// Measured: two chunks of 2048 over 18k tokens on 128 heads 4.3 ms for 5.8 TFLOP, 1.35
// PFLOP/s; 4 prompts of 2100 to 3400 tokens 1.19 ms, 1.01 PFLOP/s; 6 turns of up to 200 tokens
// 66 us. A step of both pairs of an SM takes 3000 cycles, the products' own pace, while they
// take turns at the tensor cores, and up to 4300 while both queue products and then both
// exponentials at the same time; the pairs know nothing of each other, and holding one back
// when its products took longer than they do alone gave 4 % on short chunks and lost as much
// on long ones. A tile's set-up, first copies and output cost about 12000 cycles, which
// bounds turns.
//
// Two pairs share their SMs: while one's warps turn scores into weights, copy or store, the
// tensor cores work on the other. (Two sub-tiles of one pair taking turns, with three steps'
// keys and values in flight, were as fast on long chunks, 5.48 against 5.33 ms for two chunks
// of 2048 over 18k tokens, and slower on short ones, 176 against 137 us for turns of up to
// 200: nothing overlapped a tile's set-up and output.)
//
// The pair shares the second operand: CTA r copies the keys of tokens 64 r .. 64 r + 63 of a
// step and value columns 64 r .. 64 r + 63, 40 KB a step instead of 80 KB. That halves the
// reads of L2 and takes the scores' operands (6 KB an MMA and SM, not 8) below the bandwidth
// of shared memory; with a CTA on its own the products ran at three quarters of this pace.
//
// P (bf16) is stored over the scores it came from. The products are issued in order by one
// thread of CTA 0, so that the next scores overwrite P only once P . V has read it. m is
// raised lazily, only when it grows by more than 8 (P <= 2^8).
//
// Shared memory: Q 48 KB, two steps' key blocks ([64 tokens x 64 dims] each) and a value block
// ([128 tokens x 64 columns]), copied two steps ahead (keys) and while the softmax runs
// (values). Tensor memory: S, O, 128 columns each.
// ============================================================================
constexpr int kThreads = 256;          // warp 0 copies, 1 products (CTA 0), 4..7 softmax
// Registers a thread of the first warpgroup (copies and products) and of the other (softmax)
// once they are split again: what the launch had.
constexpr int kRegsLaunch = 128, kRegsIssue = 104, kRegsSoftmax = 152;
static_assert(kRegsIssue + kRegsSoftmax <= 2 * kRegsLaunch, "register split");
constexpr int kTileQ = kPrefillTcTile;
constexpr uint32_t kKBlock = 64 * 128;                  // 8 KB
constexpr uint32_t kOffK = 3 * kBlock;                  // after Q
constexpr uint32_t kStageK = 3 * kKBlock;               // two of them
constexpr uint32_t kOffV = kOffK + 2 * kStageK;
constexpr uint32_t kOffBar = kOffV + kBlock;
constexpr uint32_t kSmemBytes = kOffBar + 128;          // (no slack: the kernel checks its base)
static_assert(kSmemBytes <= 228 * 1024 / 2 - 1024, "shared memory budget of two CTAs");
constexpr uint32_t kTmem = 256;
constexpr uint32_t kColS = 0, kColO = 128;

struct Bars {
    // of CTA 0: both CTAs' copies landed; both CTAs' weights are stored (a warp an arrival)
    uint64_t q_full, full[2], p_full;
    // of each CTA, from CTA 0's products
    uint64_t empty;            // a step's P . V is done
    uint64_t s_full;           // the step's scores are there (and the P . V before)
    uint64_t o_full;
    uint32_t tmem_base;
    int32_t abort_flag;
};
static_assert(sizeof(Bars) <= 128, "barriers");

// Pipeline timestamps for performance analysis, compiled only with -DMLA_TRACE: clock64 at
// each hand-off of CTA (0, 0) for its first kTraceSteps steps. Product builds contain none
// of it. Events: 0 turn landed, 1 weights seen, 2 P . V issued, 3 scores issued (products), 4
// scores seen, 5 maximum known, 6 weights stored (softmax)
#ifdef MLA_TRACE
constexpr int kTraceSteps = 64;
__device__ long long g_pftrace[7][kTraceSteps];
#define PTRACE(ev, step)                                                                  \
    do {                                                                                  \
        if (blockIdx.x == 0 && blockIdx.y == 0 && (step) < kTraceSteps) g_pftrace[ev][step] = clock64(); \
    } while (0)
#else
#define PTRACE(ev, step) \
    do {                 \
    } while (0)
#endif

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 2)
prefill_tc_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap rope_map,
                  const PrefillParams p, int by_seq) {
    pdl_trigger();
    pdl_wait();
    // The last tiles of a sequence see the most: they start first.
    const int tiles = p.tile_off[p.B], gave_up = p.status[1], r = (int)cluster_ctarank(), H = p.s.H;
    int b, hl, i0;
    if (by_seq) {                                        // sequence, head, tile
        const int at = blockIdx.y * (gridDim.x >> 1) + (blockIdx.x >> 1), pos = tiles * p.nh - 1 - at;
        if (pos < 0) return;                             // both CTAs of a pair
        b = find_seq(p.tile_off, p.B, pos / p.nh);
        const int off = p.tile_off[b], of_b = p.tile_off[b + 1] - off, in_b = pos - off * p.nh;
        hl = in_b / of_b;
        i0 = (in_b - hl * of_b) * kTileQ;
    } else {                                             // head, sequence, tile
        const int tile = tiles - 1 - (int)(blockIdx.x >> 1);
        if (tile < 0) return;
        b = find_seq(p.tile_off, p.B, tile);
        hl = blockIdx.y;
        i0 = (tile - p.tile_off[b]) * kTileQ;
    }
    const int h = p.h0 + hl, n = p.cu_q[b + 1] - p.cu_q[b];
    const size_t qrow0 = (size_t)p.cu_q[b] + i0;
    const int rows_here = min(kTileQ, n - i0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    __nv_bfloat16 *out = (__nv_bfloat16 *)p.out;
    extern __shared__ __align__(1024) uint8_t smem[];
    const bool misaligned = smem_u32(smem) & 1023u;      // of both CTAs: the swizzled blocks need it
    if (misaligned) raise_flag(p.status, FLAG_TIMEOUT);
    // (gave_up is the expansion's, which is complete: every thread of the pair read the same)
    if (p.bad[b] | gave_up | misaligned) {
        for (int e = r * kThreads + tid; e < rows_here * kDv; e += 2 * kThreads)
            out[((qrow0 + e / kDv) * H + h) * kDv + e % kDv] = __float2bfloat16_rn(CUDART_NAN_F);
        if (p.lse)
            for (int i = r * kThreads + tid; i < rows_here; i += 2 * kThreads) p.lse[(qrow0 + i) * H + h] = CUDART_NAN_F;
        return;
    }
    const int L = p.seq_lens[b];
    const int steps = (L - n + i0 + rows_here + 127) / 128;      // of the tile's last row
    Bars *bars = (Bars *)(smem + kOffBar);
    const int row0 = p.kv_off[b];
    const int kv0 = hl * p.cap_rows + row0;               // fits: the pass's rows are counted in 32 bits
    if (tid == 64) {                       // an idle warp: the first step's operands into L2 during the set-up
        for (int c = 0; c < 3; ++c) prefetch_3d(&q_map, 64 * c, h, (int)qrow0 + 128 * r);
        prefetch_2d(&k_map, 0, kv0 + 64 * r);
        prefetch_2d(&k_map, 64, kv0 + 64 * r);
        prefetch_2d(&rope_map, kR, row0 + 64 * r);
        prefetch_2d(&v_map, 64 * r, kv0);
    }
    if (tid == 0) {
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->full[0], 1);
        mbar_init(&bars->full[1], 1);
        mbar_init(&bars->p_full, 8);
        mbar_init(&bars->empty, 1);
        mbar_init(&bars->s_full, 1);
        mbar_init(&bars->o_full, 1);
        bars->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&bars->tmem_base)),
                     "r"(kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();                        // the other CTA's barriers and tensor memory are there
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        return mbar_wait_bounded(bar, parity, &bars->abort_flag, p.status, FLAG_TIMEOUT, kTimeoutNs);
    };

    // The copies go in turns: turn t brings step t's keys and step t - 1's values, which the
    // products take one after the other (turn 0: keys only; turn `steps`: values only). Two
    // turns are on their way at a time: turn t starts when the P . V of step t - 2 is done,
    // which read the values that stood in its place, its scores before it the keys.
    if (warp == 0) {
        // ================================================= copies
        reg_dec<kRegsIssue>();
        if (lane == 0) {
            const uint32_t q_bar = mapa(smem_u32(&bars->q_full), 0);
            if (r == 0) mbar_expect_tx(&bars->q_full, 6 * kBlock);
            for (int c = 0; c < 3; ++c)
                tma_pair_3d(smem + c * kBlock, &q_map, 64 * c, h, (int)qrow0 + 128 * r, q_bar);
            int u = 0;
            for (; u <= steps; ++u) {
                if (u > 1 && !wait(&bars->empty, u & 1)) break;
                const uint32_t bar = mapa(smem_u32(&bars->full[u & 1]), 0);
                if (r == 0) mbar_expect_tx(&bars->full[u & 1], (u < steps ? 6 * kKBlock : 0u) + (u > 0 ? 2 * kBlock : 0u));
                if (u > 0) tma_pair_2d(smem + kOffV, &v_map, 64 * r, kv0 + 128 * (u - 1), bar);
                if (u < steps) {
                    uint8_t *k = smem + kOffK + (u & 1) * kStageK;
                    tma_pair_2d(k, &k_map, 0, kv0 + 128 * u + 64 * r, bar);
                    tma_pair_2d(k + kKBlock, &k_map, 64, kv0 + 128 * u + 64 * r, bar);
                    tma_pair_2d(k + 2 * kKBlock, &rope_map, kR, row0 + 128 * u + 64 * r, bar);
                }
            }
            // Never leave a copy in flight into the pair's shared memory: CTA 0 waits here for
            // both CTAs' copies, CTA 1 for CTA 0 at the end.
            if (r == 0) {
                mbar_drain(&bars->q_full, 0);
                for (int v = max(0, u - 2); v < u; ++v) mbar_drain(&bars->full[v & 1], (v >> 1) & 1);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================================================= products: lane 0 of CTA 0 alone
        reg_dec<kRegsIssue>();
        if (lane == 0 && r == 0) {
            constexpr uint32_t kIdS = idesc_bf16(256, 128, false), kIdO = idesc_bf16(256, 128, true);
            const uint64_t qd = sdesc(smem_u32(smem), 16, 1024), kd = sdesc(smem_u32(smem + kOffK), 16, 1024);
            const uint64_t vd = sdesc(smem_u32(smem + kOffV), kBlock, 1024);                 // MN-major
            const uint32_t tS = tmem + kColS, tO = tmem + kColO;
            // Between one product and the next stand as few instructions as can be: the first
            // probe of a barrier is inline, the bounded wait out of line.
            const uint32_t full = smem_u32(bars->full), p_full = smem_u32(&bars->p_full);
            auto there = [&](uint32_t bar, uint32_t parity) {
                return mbar_test32(bar, parity) || wait_slow(bar, parity, &bars->abort_flag, p.status);
            };
            auto scores = [&](uint32_t stage) {
                const uint64_t ks = kd + stage * (kStageK >> 4);
#pragma unroll
                for (int c = 0; c < 3; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint64_t a = qd + c * (kBlock >> 4) + 2 * e, k = ks + c * (kKBlock >> 4) + 2 * e;
                        if (c == 0 && e == 0) mma2_ss<kIdS, 0>(tS, a, k);
                        else mma2_ss<kIdS, 1>(tS, a, k);
                    }
                commit2(&bars->s_full);
            };
            bool ok = wait(&bars->q_full, 0) && wait(&bars->full[0], 0);
            tc_fence_after();
            if (ok) scores(0);
            for (int j = 0; j < steps && ok; ++j) {
                const uint32_t s = (j + 1) & 1;                // of turn j + 1
                ok = there(full + 8 * s, ((j + 1) >> 1) & 1);
                PTRACE(0, j);
                ok = ok && there(p_full, j & 1);
                if (!ok) break;
                PTRACE(1, j);
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < 8; ++e) mma2_ts(tO, tS + 8 * e, vd + 128 * e, kIdO, (j > 0 || e > 0) ? 1u : 0u);
                commit2(&bars->empty);
                PTRACE(2, j);
                if (j + 1 < steps) scores(s);
                else commit2(&bars->o_full);
                PTRACE(3, j);
            }
            // products in flight must end before the tensor memory is given back
            if (!ok) commit2(&bars->o_full);
            mbar_drain(&bars->o_full, 0);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ================================================= softmax and output
        reg_inc<kRegsSoftmax>();
        const int wq = warp & 3, row = 32 * wq + lane;         // of the CTA's rows
        const int i = i0 + 128 * r + row;                      // of the sequence's new tokens
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * wq) << 16);
        const uint32_t tS = lane_addr + kColS, tO = lane_addr + kColO;
        const int seen = L - n + min(i, n - 1) + 1;            // tokens this row sees
        // where the scale is positive the maximum commutes with it: one fma per exponent
        const bool pos_scale = p.scale > 0.f;
        const float c2 = p.scale * kLog2e, cs = pos_scale ? c2 : 1.f;
        const uint32_t p_bar = mapa(smem_u32(&bars->p_full), 0);
        float m = -CUDART_INF_F, l = 0.f;
        bool ok = true;
        for (int j = 0; j < steps; ++j) {
            ok = __all_sync(0xffffffffu, wait(&bars->s_full, j & 1));
            if (!ok) break;
            tc_fence_after();
            if (tid == 128) PTRACE(4, j);
            uint32_t sv[128];
            TMEM_LD32(tS, sv);
            TMEM_LD32(tS + 32, (sv + 32));
            TMEM_LD32(tS + 64, (sv + 64));
            TMEM_LD32(tS + 96, (sv + 96));
            tmem_wait_ld();
            const int vis = seen - 128 * j;
            if (!pos_scale || __any_sync(0xffffffffu, vis < 128)) {
#pragma unroll
                for (int e = 0; e < 128; ++e) {
                    const float v = pos_scale ? __uint_as_float(sv[e]) : __uint_as_float(sv[e]) * c2;
                    sv[e] = __float_as_uint(e < vis ? v : -CUDART_INF_F);
                }
            }
            float mx[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = __uint_as_float(sv[e]);
#pragma unroll
            for (int e = 4; e < 128; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(sv[e]));
            const float m_new = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * cs);
            if (tid == 128) PTRACE(5, j);
            float alpha = 1.f;
            bool rescale = false;
            if (m_new > m + 8.f) {
                alpha = exp2f(m - m_new);                      // 0 at the first step
                m = m_new;
                rescale = j > 0;
            }
            const float nm = m == -CUDART_INF_F ? -CUDART_INF_F : -m;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 64; ++e) {
                const float x = ex2(fmaf(__uint_as_float(sv[2 * e]), cs, nm));
                const float y = ex2(fmaf(__uint_as_float(sv[2 * e + 1]), cs, nm));
                const __nv_bfloat162 w = __floats2bfloat162_rn(x, y);
                sum[(2 * e) & 3] += x;             // unrounded: the denominator does not see P's rounding
                sum[(2 * e + 1) & 3] += y;
                sv[e] = *(const uint32_t *)&w;
            }
            l = l * alpha + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
            // the scores' barrier says that the P . V before is done as well
            if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t ov[32];
                    TMEM_LD32(tO + 32 * c, ov);
                    tmem_wait_ld(ov);
#pragma unroll
                    for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                    TMEM_ST32(tO + 32 * c, ov);
                }
            }
            TMEM_ST32(tS, sv);
            TMEM_ST32(tS + 32, (sv + 32));
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(p_bar);
            if (tid == 128) PTRACE(6, j);
        }
        ok = ok && __all_sync(0xffffffffu, wait(&bars->o_full, 0));
        ok = ok && __all_sync(0xffffffffu, *(volatile int32_t *)&bars->abort_flag == 0);
        tc_fence_after();
        // O / l through this warp's part of the Q blocks (read for the last time by the last
        // scores), then rows of 256 bytes
        uint8_t *stage = smem + wq * 32 * 256;
        const float inv = ok ? 1.f / l : CUDART_NAN_F;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            uint32_t ov[32];
            TMEM_LD32(tO + 32 * c, ov);
            tmem_wait_ld(ov);
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(ov[8 * ch + 2 * e]) * inv,
                                                                   __uint_as_float(ov[8 * ch + 2 * e + 1]) * inv);
                    w[e] = *(const uint32_t *)&x;
                }
                // 16-byte chunks rotated by the row: no two lanes of a store on one bank
                *(uint4 *)(stage + lane * 256 + (((4 * c + ch) ^ (lane & 15)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        __syncwarp();
        const int first = 128 * r + 32 * wq;                   // of the tile
        for (int rr = lane >> 4; rr < 32; rr += 2)
            if (first + rr < rows_here)
                *(uint4 *)(out + ((qrow0 + first + rr) * H + h) * kDv + 8 * (lane & 15)) =
                    *(const uint4 *)(stage + rr * 256 + (((lane & 15) ^ (rr & 15)) << 4));
        if (p.lse && first + lane < rows_here)
            p.lse[(qrow0 + first + lane) * H + h] = ok ? (m + log2f(l)) * kLn2 : CUDART_NAN_F;
    } else {
        reg_dec<kRegsIssue>();
    }
    // neither CTA leaves while the other may reach its barriers, its shared memory or its
    // tensor memory
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
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

// bf16 map over a row-major [rows, cols] matrix, 128-byte swizzled boxes of [box_rows, 64].
// Loads past the last row read zeros.
static bool map2d(CUtensorMap *map, const void *base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
    cuuint32_t box[2] = {64, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The query [num_q, H, 192], boxes of 128 tokens x 64 dims of one head.
static bool map_q(CUtensorMap *map, const void *base, int num_q, int H) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t d = kDn + kRope;
    cuuint64_t dims[3] = {d, (cuuint64_t)H, (cuuint64_t)num_q};
    cuuint64_t strides[2] = {d * 2, d * 2 * (cuuint64_t)H};
    cuuint32_t box[3] = {64, 1, 128};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace pf

bool prefill_tc_supported(const ShapeArgs &s, int dn) {
    return (s.kind == MLA_KV_BF16 || is_mx(s.kind)) && s.r == pf::kR && s.dR == pf::kRope && s.dv == pf::kDv && dn == pf::kDn;
}

cudaError_t launch_prefill_tc(const PrefillParams &p, cudaStream_t st) {
    using namespace pf;
    const uint64_t kv_rows = (uint64_t)p.nh * p.cap_rows;
    CUtensorMap rows, uk, uv, q, k_ld, v_ld, rope;
    if (!map2d(&rows, p.rows, p.cap_rows, kR + kRope, 128) || !map2d(&uk, p.W_UK, (uint64_t)p.s.H * kDn, kR, 128) ||
        !map2d(&uv, p.W_UV, (uint64_t)p.s.H * kR, kDv, 64) || !map2d(&k_ld, p.k, kv_rows, kDn, 64) ||
        !map2d(&v_ld, p.v, kv_rows, kDv, 128) || !map2d(&rope, p.rows, p.cap_rows, kR + kRope, 64) || !map_q(&q, p.q, p.num_q, p.s.H))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(ex::expand_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ex::kSmemBytes);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(prefill_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    // the register split draws on what the launch has: refuse a build that has less
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, prefill_tc_kernel);
    if (e != cudaSuccess) return e;
    if (at.numRegs < kRegsLaunch) return cudaErrorInvalidConfiguration;
    // Heads a pair of CTAs makes in a row: those that give the least rounds x (heads + what a
    // pair's start and end cost, about 2.5 heads' time). The rows that the sequences' ends
    // leave of their last 128 are counted half.
    int dev = 0, sms = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return e;
    const long long tiles = (p.cap_rows + 255) / 256, likely = (p.cap_rows - 64ll * p.B + 255) / 256;
    long long heads = 2, least = LLONG_MAX;
    for (int n = 2; n < p.nh + 2; n += 2) {
        const long long cost = (2 * n + 5) * ((likely * ((p.nh + n - 1) / n) + sms / 2 - 1) / (sms / 2));
        if (cost < least) {
            least = cost;
            heads = n;
        }
    }
    e = launch_pdl(ex::expand_tc_kernel, dim3((unsigned)(2 * tiles), (unsigned)((p.nh + heads - 1) / heads)), dim3(ex::kThreads),
                   ex::kSmemBytes, st, rows, uk, uv, p, (int)heads);
    if (e != cudaSuccess) return e;
    // The order of the tiles. Head by head the heaviest sequence's tiles are among the last to
    // start too, so where there are few rounds the sequences go one after the other instead: 8
    // chunks of 1025 to 1992 tokens on 16 heads (6 rounds of the pairs that fit) 439 us instead
    // of 464, 8 of 256 on 64 heads (3) 266 instead of 272, but 4 prompts on 128 heads (37) 1452
    // instead of 1443, 8 chunks of 768 on 64 heads (10) 534 instead of 529. Between them it
    // depends on the lengths, and the border is low: chunks of 1000 to 2000 tokens gain 3.9 % at
    // 9 rounds, 2.3 % at 14; prompts of 1000 to 4000 1.9 % at 9, 0.6 % at 19; chunks of 1 to 1500
    // 1.4 % at 16, 1.0 % at 21, 0.3 % at 32.
    const int pairs = p.num_q / kTileQ + p.B, by_seq = (long long)pairs * p.nh < 8ll * sms;
    return launch_pdl(prefill_tc_kernel, dim3(2 * pairs, p.nh), dim3(kThreads), kSmemBytes, st, q, k_ld, v_ld, rope, p, by_seq);
}

}  // namespace mla

#ifdef MLA_TRACE
extern "C" int mla_prefill_trace_read(long long *events) {
    return (int)cudaMemcpyFromSymbol(events, mla::pf::g_pftrace, sizeof(mla::pf::g_pftrace));
}
#endif
