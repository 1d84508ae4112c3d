// Which drafted tokens stand, and the token that follows them (mla_draft_accept).
//
// Draft i stands if u_i q_i(x_i) < p_i(x_i). The product of two fp32 values is exact in
// fp64, so this decision is the definition's own. Behind the n drafts that stand, the next
// token has the weights w_j = max(p_n(j) - q_n(j), 0) (p_n(j) where all drafts stood), and is
// the first j whose sum w_0 + .. + w_j is above v times the sum of all. Where that is depends
// on sums over the whole vocabulary: weights are held as whole numbers of 2^-62 (a
// probability's 24 bits shifted; what is below 2^-62 is cut off) and added in 64 bits, so
// that a sum is the same in any order and every split of a row gives the same token.
//
// A row of target and draft probabilities is read once, by a warp a contiguous part; then
// the part that holds the token is read again.
#include "mla_internal.cuh"

#include <cooperative_groups.h>

namespace cg = cooperative_groups;

namespace mla {
namespace {

typedef unsigned long long u64;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kUnroll = 8;                   // loads of a lane in flight, of each row

enum Weights { kPlain, kRest, kWithout };    // p; max(p - q, 0); p without one token

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ u64 units(float v) { return __float2ull_rz(v * 0x1p62f); }
__device__ __forceinline__ bool is_probability(float v) { return v >= 0.f && v <= 1.f; }

template <Weights W, typename T>
__device__ __forceinline__ u64 weight(T p, T q, bool out) {
    if (W == kWithout && out) return 0;
    const u64 a = units(widen(p));
    if (W != kRest) return a;
    const u64 b = units(widen(q));
    return a > b ? a - b : 0;
}

struct Shared {
    u64 warp[kWarps], scan[33], sum;
    float warp_p[kWarps], sum_p;             // of the target's probabilities
    int bad, n;
};

// A warp's sums over [lo, hi) of a row.
template <Weights W, typename T>
__device__ __forceinline__ u64 sum_part(const T *p, const T *q, int x, int lo, int hi, float &sum_p, bool &bad) {
    u64 s = 0;
    for (int i0 = lo + (threadIdx.x & 31); i0 < hi; i0 += 32 * kUnroll) {
        T a[kUnroll], b[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const bool in = i0 + 32 * k < hi;
            a[k] = in ? p[i0 + 32 * k] : (T)0.f;
            b[k] = W == kRest && in ? q[i0 + 32 * k] : (T)0.f;
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            s += weight<W>(a[k], b[k], i0 + 32 * k == x);
            sum_p += widen(a[k]);
            bad |= !is_probability(widen(a[k])) || !is_probability(widen(b[k]));
        }
    }
    return s;
}

// The token of [lo, hi) at which the sum that starts at `base` passes t. Called by a whole
// block, of which one thread writes it.
template <Weights W, typename T>
__device__ __forceinline__ void find_token(const T *p, const T *q, int x, int lo, int hi, u64 base, u64 t, u64 *scan,
                                           int32_t *token) {
    const int each = (hi - lo + kThreads - 1) / kThreads;
    const int a = min(hi, lo + (int)threadIdx.x * each), e = min(hi, a + each);
    u64 s = 0, all;
    for (int i = a; i < e; ++i) s += weight<W>(p[i], W == kRest ? q[i] : (T)0.f, i == x);
    u64 at = base + block_exclusive_scan(s, scan, all);
    if (t < at || t >= at + s) return;
    for (int i = a; i < e; ++i) {
        at += weight<W>(p[i], W == kRest ? q[i] : (T)0.f, i == x);
        if (at > t) {
            *token = i;
            return;
        }
    }
}

// A cluster of CTAs a sequence, each with a part of the row.
template <typename T>
__global__ void __launch_bounds__(kThreads) accept_kernel(const AcceptParams a) {
    __shared__ Shared sh;
    const cg::cluster_group cl = cg::this_cluster();
    const int rank = cl.block_rank(), C = cl.num_blocks();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x / C, K = a.K, V = a.V;
    pdl_wait();
    pdl_trigger();
    const int k = a.counts ? a.counts[b] : K;
    const int len = a.lens ? a.lens[b] : K;
    const int32_t *x = a.x + (size_t)b * K;
    const float *u = a.u + (size_t)b * (K + 1);
    int32_t *tokens = a.tokens + (size_t)b * (K + 1);
    const bool short_len = len < K && k >= 0;
    bool bad = k > K || short_len;
    if (tid == 0) {
        sh.n = bad ? 0 : k;
        sh.bad = 0;
    }
    __syncthreads();
    if (!bad && k >= 0) {
        if (tid < k) {
            const int xi = x[tid];
            const float ui = u[tid];
            if (xi >= 0 && xi < V) {
                const float p = widen(((const T *)a.p)[((size_t)b * (K + 1) + tid) * a.p_stride + xi]);
                const float q = a.q ? widen(((const T *)a.q)[((size_t)b * K + tid) * a.q_stride + xi]) : 1.f;
                if (!is_probability(p) || !is_probability(q) || !is_probability(ui)) sh.bad = 1;
                if (!((double)ui * (double)q < (double)p)) atomicMin(&sh.n, tid);
            } else {
                sh.bad = 1;
            }
        }
        if (tid == 0 && !is_probability(u[K])) sh.bad = 1;
    }
    __syncthreads();
    bad |= sh.bad != 0;
    const int n = sh.n;
    int token_by = -1;                       // the CTA that finds the token
    u64 total = 0, base = 0, t = 0;
    const T *p = (const T *)a.p + ((size_t)b * (K + 1) + max(n, 0)) * a.p_stride;
    const T *q = nullptr;
    int w = kPlain, out = -1;
    // 32 tokens at a time, evenly over the warps of all CTAs
    const int64_t groups = (V + 31ll) / 32, warps = (int64_t)C * kWarps;
    const auto edge = [&](int64_t i) { return (int)min((int64_t)V, groups * i / warps * 32); };
    if (!bad && k >= 0) {
        if (n < k) {
            w = a.q ? kRest : kWithout;
            if (a.q) q = (const T *)a.q + ((size_t)b * K + n) * a.q_stride;
            else out = x[n];
        }
        for (;;) {
            const int64_t at = (int64_t)rank * kWarps + warp;
            const int lo = edge(at), hi = edge(at + 1);
            float sum_p = 0.f;
            bool odd = false;
            u64 s = w == kRest ? sum_part<kRest>(p, q, out, lo, hi, sum_p, odd)
                    : w == kWithout ? sum_part<kWithout>(p, q, out, lo, hi, sum_p, odd)
                                    : sum_part<kPlain>(p, q, out, lo, hi, sum_p, odd);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            sum_p = warp_sum(sum_p);
            if (lane == 0) {
                sh.warp[warp] = s;
                sh.warp_p[warp] = sum_p;
            }
            if (odd) sh.bad = 1;
            __syncthreads();
            if (tid == 0) {
                u64 all = 0;
                float all_p = 0.f;
                for (int i = 0; i < kWarps; ++i) {
                    all += sh.warp[i];
                    all_p += sh.warp_p[i];
                }
                sh.sum = all;
                sh.sum_p = all_p;
            }
            cl.sync();
            total = 0;
            sum_p = 0.f;
            int odd_row = 0;
            for (int c = 0; c < C; ++c) {
                const Shared *o = cl.map_shared_rank(&sh, c);
                if (c == rank) base = total;
                total += o->sum;
                sum_p += o->sum_p;
                odd_row |= o->bad;
            }
            cl.sync();                       // (also: nobody's numbers are read any longer)
            // probabilities add up to one; up to two, sums of units stay below 2^63
            bad = odd_row || !(sum_p <= 2.f) || (total == 0 && w == kPlain);
            if (bad || total > 0) break;
            w = kPlain;                      // nothing is left of p - q: p itself
            out = -1;
        }
        if (!bad) {
            const float v = u[K];            // t = floor(v total); for 1 the last token that has any weight
            t = v < 1.f ? __umul64hi(__float2ull_rz(v * 0x1p64f), total) : total - 1;
            token_by = t >= base && t < base + sh.sum ? rank : -1;
        }
    } else {
        cl.sync();                           // new_lens may be seq_lens: every CTA has read the length
    }
    if (rank == 0) {
        const int stand = bad || k < 0 ? 0 : n;
        for (int i = tid; i <= K; i += kThreads)
            if (bad || k < 0 || i != n) tokens[i] = i < stand ? x[i] : -1;
        if (tid == 0) {
            a.accepted[b] = stand;
            if (a.new_lens) a.new_lens[b] = k < 0 || short_len ? len : len - K + stand;
            if (bad) raise_flag(a.status, short_len ? FLAG_BAD_LENGTH : FLAG_BAD_VALUE);
        }
    }
    if (token_by != rank) return;
    u64 from = base;
    int i = 0;
    for (; i < kWarps - 1 && t >= from + sh.warp[i]; ++i) from += sh.warp[i];
    const int lo = edge((int64_t)rank * kWarps + i), hi = edge((int64_t)rank * kWarps + i + 1);
    if (w == kRest) find_token<kRest>(p, q, out, lo, hi, from, t, sh.scan, tokens + n);
    else if (w == kWithout) find_token<kWithout>(p, q, out, lo, hi, from, t, sh.scan, tokens + n);
    else find_token<kPlain>(p, q, out, lo, hi, from, t, sh.scan, tokens + n);
}

template <typename T>
cudaError_t launch(const AcceptParams &p, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    const unsigned C = 1;
    cfg.gridDim = dim3((unsigned)p.B * C);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, accept_kernel<T>, p);
}

}  // namespace

cudaError_t launch_accept(const AcceptParams &p, bool bf16, cudaStream_t st) {
    return bf16 ? launch<__nv_bfloat16>(p, st) : launch<float>(p, st);
}

}  // namespace mla
