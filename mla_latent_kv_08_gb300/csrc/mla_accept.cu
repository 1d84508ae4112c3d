// Which drafted tokens stand, and the token that follows them (mla_draft_accept).
//
// Draft i stands if u_i q_i(x_i) < p_i(x_i). The product of two fp32 values is exact in
// fp64, so this decision is the definition's own. Behind the n drafts that stand, the next
// token has the weights w_j = max(p_n(j) - q_n(j), 0) (p_n(j) where all drafts stood), and is
// the first j whose sum w_0 + .. + w_j is above v times the sum of all. Where that is depends
// on sums over the whole vocabulary: probabilities are held as whole numbers of 2^-46 (exact
// from 2^-23 on, rounded to nearest below) and added in 64 bits, so that a sum is the same in
// any order, and every split of a row gives the same token. Over 131072 tokens the roundings
// move a border by about 2^-39 of the row's weight.
//
// A row of target and draft probabilities is read once, by a warp a contiguous part, split
// over a cluster of CTAs; then the part that holds the token is read again. A call is bound by
// its chain of dependent steps (the drafts, their probabilities, the row, the cluster's sums, the
// token: 4.1 us for 500 tokens) and, for a batch, by memory in the middle of it: a lane has 32 loads of
// each row in flight. 32 sequences of 131072 tokens: 10.8 us, of which the rows take 4.6 at 6.0 TB/s
// (8 loads of each row: 15.7; 78 us with a CTA a sequence and conversions to 64 bits in hardware). One
// sequence of 32000: 4.7 us (19.5); 64 of 50257 in bf16, drafts given: 7.2 us (19.4).
#include "mla_internal.cuh"

#include <cooperative_groups.h>

#include <utility>

namespace cg = cooperative_groups;

namespace mla {
namespace {

typedef unsigned long long u64;
constexpr int kThreads = 256, kWarps = kThreads / 32;   // (512: 5.3 us at 2000 tokens, 1024: 7.3)
constexpr int kMaxCluster = 16;
constexpr int kGroup = 1024;                 // tokens that a warp takes at a time

enum Weights { kPlain, kRest, kWithout };    // p; max(p - q, 0); p without one token

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ bool is_probability(float v) { return v >= 0.f && v <= 1.f; }

// v in [0, 1] as round(v 2^46) = 2^23 hi + lo (and a constant each): v + 1 has the multiples of 2^-23
// as its last bits, and what that rounding leaves, exact, plus 1.5 2^-23 those of 2^-46. Four
// additions; shifting the 24 bits of v to their place by the exponent took three times as long.
struct Fixed {
    int hi, lo;
};
constexpr int kHi = 0x3f800000, kLo = 0x34400000;        // the bits of 1 and of 1.5 2^-23
__device__ __forceinline__ Fixed fixed(float v) {
    const float a = __fadd_rn(v, 1.f), rest = __fsub_rn(v, __fsub_rn(a, 1.f));
    return {__float_as_int(a), __float_as_int(__fadd_rn(rest, __int_as_float(kLo)))};
}
__device__ __forceinline__ u64 units(int hi, int lo) { return (u64)(((long long)hi << 23) + lo); }

// A weight, without its constants: max(p - q, 0), p, or nothing.
template <Weights W, typename T>
__device__ __forceinline__ Fixed weight(T p, T q, bool out) {
    const Fixed a = fixed(widen(p));
    if (W == kRest) {
        const Fixed b = fixed(widen(q));
        return widen(p) > widen(q) ? Fixed{a.hi - b.hi, a.lo - b.lo} : Fixed{0, 0};
    }
    return W == kWithout && out ? Fixed{0, 0} : Fixed{a.hi - kHi, a.lo - kLo};
}

// floor(v total), v in [0, 1): v's bits down to 2^-64, below 2^-17 those down to 2^-81, which are all
// of v from 2^-57 on; total is below 2^49, so that for less it is 0.
__device__ __forceinline__ u64 share(float v, u64 total) {
    return v < 0x1p-17f ? __umul64hi(__float2ull_rz(v * 0x1p81f), total) >> 17 : __umul64hi(__float2ull_rz(v * 0x1p64f), total);
}

// What a CTA found in its part of a row, and what every CTA finds for itself: whether anything
// is wrong, how many drafts stand and which weights come behind them (below 0: left out).
struct Part {
    u64 sum;
    float p;                                 // sum of the target's probabilities
    int bad, found;
};
struct Shared {
    Part all[2][kMaxCluster];                // of every CTA of the cluster, by pass
    u64 warp[kWarps], scan[33];
    float warp_p[kWarps];
    int bad, n;
};

// A warp's sums over [lo, hi) of a row; `bad` is set where this lane saw what is no probability. In the
// order of their bits as whole numbers, negative values and NaN come behind 1; only -0 has to
// be told from them, where there is anything to tell.
template <Weights W, typename T>
__device__ __forceinline__ u64 sum_part(const T *p, const T *q, int x, int lo, int hi, float &sum_p, bool &bad) {
    u64 s = 0;
    int hi_sum = 0, lo_sum = 0;              // of a few weights
    uint32_t most = 0;
    const auto add = [&](T a, T b, int i) {
        const Fixed w = weight<W>(a, b, i == x);
        hi_sum += w.hi;
        lo_sum += w.lo;
        sum_p += widen(a);
        most = max(most, max(__float_as_uint(widen(a)), __float_as_uint(widen(b))));
    };
    int i0 = lo + (threadIdx.x & 31);
    for (; i0 + kGroup - 32 < hi; i0 += kGroup) {
        T a[kGroup / 32], b[kGroup / 32];
#pragma unroll
        for (int k = 0; k < kGroup / 32; ++k) {
            a[k] = p[i0 + 32 * k];
            b[k] = W == kRest ? q[i0 + 32 * k] : (T)0.f;
        }
#pragma unroll
        for (int k = 0; k < kGroup / 32; ++k) add(a[k], b[k], i0 + 32 * k);
        s += units(hi_sum, lo_sum);
        hi_sum = lo_sum = 0;
    }
#pragma unroll 4
    for (; i0 < hi; i0 += 32) add(p[i0], W == kRest ? q[i0] : (T)0.f, i0);
    s += units(hi_sum, lo_sum);
    if (most > 0x3f800000u)
        for (int i = lo + (threadIdx.x & 31); i < hi; i += 32)
            bad |= !is_probability(widen(p[i])) || (W == kRest && !is_probability(widen(q[i])));
    return s;
}

// The token of [lo, hi) at which the sum that starts at `base` passes t. Called by a whole
// block, of which one thread writes it.
template <Weights W, typename T>
__device__ __forceinline__ void find_token(const T *p, const T *q, int x, int lo, int hi, u64 base, u64 t, u64 *scan,
                                           int32_t *token) {
    constexpr int kEach = 8;
    for (int i0 = lo; i0 < hi; i0 += kEach * kThreads) {
        const int i = i0 + kEach * (int)threadIdx.x;
        u64 v[kEach], s = 0, all;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const Fixed f = i + k < hi ? weight<W>(p[i + k], W == kRest ? q[i + k] : (T)0.f, i + k == x) : Fixed{0, 0};
            v[k] = units(f.hi, f.lo);
            s += v[k];
        }
        u64 at = base + block_exclusive_scan(s, scan, all);
        base += all;
        if (t >= base) continue;             // for the whole block: not among these
        if (t < at || t >= at + s) return;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            if (t >= at && t < at + v[k]) *token = i + k;
            at += v[k];
        }
        return;
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
    const int32_t *x = a.x + (size_t)b * K;
    const float *u = a.u + (size_t)b * (K + 1);
    // these loads wait for nothing
    const int xi = tid < K ? x[tid] : 0;
    const float ui = tid < K ? u[tid] : 0.f, v = u[K];
    const int k = a.counts ? a.counts[b] : K;
    const int len = a.lens ? a.lens[b] : K;
    // new_lens may be seq_lens: no CTA writes before all have read. (And a CTA's shared memory
    // is there once it has begun.)
    auto here = cl.barrier_arrive();
    int32_t *tokens = a.tokens + (size_t)b * (K + 1);
    const bool short_len = len < K && k >= 0;
    bool bad = k > K || short_len;
    if (tid == 0) {
        sh.n = bad ? 0 : max(k, 0);
        sh.bad = 0;
    }
    __syncthreads();
    if (!bad && k >= 0) {
        if (tid < k) {
            if (xi >= 0 && xi < V) {
                const float p = widen(((const T *)a.p)[((size_t)b * (K + 1) + tid) * a.p_stride + xi]);
                const float q = a.q ? widen(((const T *)a.q)[((size_t)b * K + tid) * a.q_stride + xi]) : 1.f;
                if (!is_probability(p) || !is_probability(q) || !is_probability(ui)) sh.bad = 1;
                if (!((double)ui * (double)q < (double)p)) atomicMin(&sh.n, tid);
            } else {
                sh.bad = 1;
            }
        }
        if (tid == 0 && !is_probability(v)) sh.bad = 1;
    }
    __syncthreads();
    bad |= sh.bad != 0;
    const int n = sh.n;
    bool mine = false, left_out = false;     // this CTA's part has the token; the sequence has none
    u64 total = 0, base = 0, own = 0, t = 0;
    const T *p = (const T *)a.p + ((size_t)b * (K + 1) + n) * a.p_stride;
    const T *q = nullptr;
    int w = kPlain, out = -1;
    const bool reads = !bad && k >= 0;
    if (reads && n < k) {
        w = a.q ? kRest : kWithout;
        if (a.q) q = (const T *)a.q + ((size_t)b * K + n) * a.q_stride;
        else out = x[n];
    }
    // evenly over the warps of all CTAs, a group of tokens at a time where there are so many
    const unsigned warps = C * kWarps, group = V >= kGroup * (int64_t)warps ? kGroup : 32;
    const unsigned each = ((V + group - 1) / group + warps - 1) / warps * group;         // tokens of a warp
    const auto edge = [&](int i) { return (int)min((int64_t)V, (int64_t)i * each); };
    cl.barrier_wait(std::move(here));
    for (int pass = 0;; ++pass) {
        const int at = rank * kWarps + warp;
        const int lo = edge(at), hi = reads ? edge(at + 1) : lo, found = k < 0 ? -1 : 4 * n + w;
        float sum_p = 0.f;
        bool odd = bad;
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
        if (tid < C) {                       // every CTA tells every other
            Part part = {0, 0.f, sh.bad, found};
            for (int i = 0; i < kWarps; ++i) {
                part.sum += sh.warp[i];
                part.p += sh.warp_p[i];
            }
            cl.map_shared_rank(&sh, tid)->all[pass][rank] = part;
        }
        cl.sync();
        // from here on all CTAs go the same way, whatever else: should they have found different
        // things (inputs that another stream changes meanwhile), the sequence is refused
        // lane c looks at CTA c's part
        const Part part = lane < C ? sh.all[pass][lane] : Part{0, 0.f, 0, 0};
        const bool odd_row = __any_sync(0xffffffffu, lane < C && (part.bad || part.found != sh.all[pass][0].found));
        sum_p = warp_sum(part.p);
        u64 upto = part.sum;
#pragma unroll
        for (int o = 1; o < kMaxCluster; o <<= 1) {
            const u64 v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        total = __shfl_sync(0xffffffffu, upto, kMaxCluster - 1);
        own = __shfl_sync(0xffffffffu, part.sum, rank);
        base = __shfl_sync(0xffffffffu, upto, rank) - own;
        // probabilities add up to one, at most to two. Their sum here is an fp32 one, whose order follows
        // from the split: a lane's additions, 2^22 at most, each round up by at most 2^-24 of a sum, a
        // quarter of it in all. So what adds up to two is never refused, and whole numbers stay below 2^49
        left_out = !odd_row && found < 0;
        bad = odd_row || !(sum_p <= 2.5f) || (total == 0 && w == kPlain && !left_out);
        if (bad || left_out || total > 0) break;
        w = kPlain;                          // nothing is left of p - q: p itself
        out = -1;
    }
    if (!bad && !left_out) {                 // t = floor(v total); for 1 the last token that has any weight
        t = v < 1.f ? share(v, total) : total - 1;
        mine = t >= base && t < base + own;
    }
    if (rank == 0) {
        const bool none = bad || left_out;
        const int stand = none ? 0 : n;
        for (int i = tid; i <= K; i += kThreads)
            if (none || i != n) tokens[i] = i < stand ? x[i] : -1;
        if (tid == 0) {
            a.accepted[b] = stand;
            if (a.new_lens) a.new_lens[b] = left_out || short_len ? len : len - K + stand;
            if (bad) raise_flag(a.status, short_len ? FLAG_BAD_LENGTH : FLAG_BAD_VALUE);
        }
    }
    if (!mine) return;
    // the warp whose part has it: the last of those that begin at or before t
    u64 from = lane < kWarps ? sh.warp[lane] : 0;
    const u64 its = from;
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
        const u64 v = __shfl_up_sync(0xffffffffu, from, o);
        if (lane >= o) from += v;
    }
    from += base - its;
    const int i = 31 - __clz(__ballot_sync(0xffffffffu, lane < kWarps && from <= t));
    from = __shfl_sync(0xffffffffu, from, i);
    const int lo = edge(rank * kWarps + i), hi = edge(rank * kWarps + i + 1);
    if (w == kRest) find_token<kRest>(p, q, out, lo, hi, from, t, sh.scan, tokens + n);
    else if (w == kWithout) find_token<kWithout>(p, q, out, lo, hi, from, t, sh.scan, tokens + n);
    else find_token<kPlain>(p, q, out, lo, hi, from, t, sh.scan, tokens + n);
}

// CTAs a sequence: a power of two up to 8 (odd numbers are slower than the next lower one), with 1024
// tokens each at least, and two CTAs an SM at most: a second round of clusters costs more than the split
// gives (an fp32 row and a draft's: 32 sequences of 50257 tokens 7.3 us with 8 and 8.5 with 4, 40 11.2 and
// 9.4; 72 of 32000 7.6 with 4 and 8.4 with 2, 80 10.1 and 9.3; 190 14.6 with 2, 14.4 with 1). Parts of 32768 tokens and more are halved up to 2.75 CTAs an SM, since the halves spread
// over the SMs (52 of 200000: 23.9 with 8, 26.0 with 4; 104: 38.6 with 4, 45.4 with 2). Few sequences
// get 16 (12 of 131072: 6.8 with 16, 8.2 with 8; 20: 10.3, 9.2), as long as that is 4 CTAs for 3 SMs.
// No limit is the best one for every length: 220 of 200000 take 83.3 with the 1 of this rule, 63.1
// with 4; 160 of 32000 13.8 with its 1, 11.8 with 2; 40 of 129280 14.4 with its 4, 13.4 with 8; 20 of
// 200000 13.9 with its 8, 13.4 with 16.
unsigned cluster_size(int32_t B, int32_t V, int32_t sms) {
    const unsigned most = 16ll * B <= 4 * sms / 3 ? 16 : 8;
    unsigned C = 1;
    while (C < most && 1024ll * C < V && 2 * C * (int64_t)B <= ((unsigned)V / C < 32768 ? 2 * sms : 11 * sms / 4)) C *= 2;
    return C;
}

template <typename T>
cudaError_t launch(const AcceptParams &p, cudaStream_t st) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const unsigned C = cluster_size(p.B, p.V, sms);
    if (C > 8) {
        e = cudaFuncSetAttribute(accept_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.B * C);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, accept_kernel<T>, p);
}

}  // namespace

cudaError_t launch_accept(const AcceptParams &p, bool bf16, cudaStream_t st) {
    return bf16 ? launch<__nv_bfloat16>(p, st) : launch<float>(p, st);
}

}  // namespace mla
