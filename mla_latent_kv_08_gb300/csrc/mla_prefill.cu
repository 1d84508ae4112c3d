// Prefill on the CUDA cores, for every shape, and the plan that both prefill paths use.
//
// With c_t a cached token's latent and kR_t its rope key, per head h:
//   k_t = [W_UK[h] c_t ; kR_t],  v_t = W_UV[h]^T c_t,
//   out_i = sum_{t visible to i} softmax_t(scale q_i . k_t) v_t.
// The plan gives every sequence a run of dense rows; the cache is read into them once;
// then, for as many heads at a time as the workspace holds, keys and values are made and
// attended over with a running maximum and sum.
#include "mla_internal.cuh"

#include <math_constants.h>

namespace mla {

// Block-wide exclusive scan of a 64-bit value; `total` to all.
__device__ __forceinline__ long long scan_block(long long v, long long *s_warp, long long &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    long long before = 0, all = 0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) {
        const long long x = s_warp[w];
        if (w < warp) before += x;
        all += x;
    }
    total = all;
    __syncthreads();
    return before + incl - v;
}

__global__ void __launch_bounds__(1024) prefill_plan_kernel(PrefillParams p) {
    __shared__ long long s_warp[32];
    pdl_trigger();
    if (threadIdx.x == 0) {
        p.status[0] = p.gave_up ? FLAG_TIMEOUT : 0;
        p.status[1] = p.gave_up;
    }
    __syncthreads();
    const long long cap_tokens = (long long)p.max_blocks * p.s.bs;
    long long rows0 = 0, tiles0 = 0;
    for (int base = 0; base < p.B; base += blockDim.x) {
        const int b = base + threadIdx.x;
        long long rows = 0, tiles = 0;
        bool bad = false;
        if (b < p.B) {
            const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], L = p.seq_lens[b];
            if (q0 < 0 || q1 < q0 || q1 > p.num_q) {
                bad = true;                            // no rows of this sequence can be told
            } else if (q1 > q0) {
                tiles = (q1 - q0 + p.tile_q - 1) / p.tile_q;
                bad = L < q1 - q0 || L > cap_tokens;
                if (!bad) rows = ((long long)L + 127) / 128 * 128;
            }
        }
        long long tot_rows, tot_tiles;
        const long long r0 = rows0 + scan_block(rows, s_warp, tot_rows);
        const long long t0 = tiles0 + scan_block(tiles, s_warp, tot_tiles);
        if (b < p.B) {
            bad = bad || r0 + rows > p.cap_rows;
            p.kv_off[b] = (int)min(r0, (long long)p.cap_rows);
            p.tile_off[b] = (int)t0;
            p.bad[b] = bad ? 1 : 0;
            if (bad) raise_flag(p.status, FLAG_BAD_LENGTH);
        }
        rows0 += tot_rows;
        tiles0 += tot_tiles;
    }
    if (threadIdx.x == 0) {
        p.kv_off[p.B] = (int)min(rows0, (long long)p.cap_rows);
        p.tile_off[p.B] = (int)tiles0;
    }
}

cudaError_t launch_prefill_plan(const PrefillParams &p, cudaStream_t st) {
    prefill_plan_kernel<<<1, p.B >= 1024 ? 1024 : (p.B + 31) / 32 * 32, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// y[h][row][j] = sum_k rows[row][k] W[h][j][k] (W_UK: K-major) or W[h][k][j] (W_UV), fp32.
// A CTA makes a 64 x 64 tile; thread (ty, tx) a 4 x 4 block. A latent with a NaN or an
// infinity gives NaN keys, so that every new token that sees it is NaN, and zero values, so
// that those whose mask hides it (weight 0) are as if it were not there.
template <typename T, bool UK>
__global__ void __launch_bounds__(256) expand_simt_kernel(PrefillParams p) {
    __shared__ float sA[32][64 + 1], sB[32][64 + 1];
    const int r = p.s.r, D = p.s.D(), N = UK ? p.dn : p.s.dv;
    const int m0 = blockIdx.x * 64, j0 = blockIdx.y * 64, h = p.h0 + blockIdx.z;
    if (m0 >= p.kv_off[p.B]) return;
    const T *rows = (const T *)p.rows;
    const T *W = (const T *)(UK ? p.W_UK : p.W_UV) + (size_t)h * r * N;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < r; k0 += 32) {
        for (int e = threadIdx.x; e < 64 * 32; e += 256) {
            const int m = e >> 5, kk = e & 31;          // rows: consecutive lanes along k
            sA[kk][m] = k0 + kk < r ? to_f32(rows[(size_t)(m0 + m) * D + k0 + kk]) : 0.f;
            if (UK) sB[kk][m] = (k0 + kk < r && j0 + m < N) ? to_f32(W[(size_t)(j0 + m) * r + k0 + kk]) : 0.f;
        }
        if (!UK)
            for (int e = threadIdx.x; e < 64 * 32; e += 256) {
                const int j = e & 63, kk = e >> 6;
                sB[kk][j] = (k0 + kk < r && j0 + j < N) ? to_f32(W[(size_t)(k0 + kk) * N + j0 + j]) : 0.f;
            }
        __syncthreads();
#pragma unroll 4
        for (int kk = 0; kk < 32; ++kk) {
            float a[4], b[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                a[u] = sA[kk][4 * ty + u];
                b[u] = sB[kk][4 * tx + u];
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(a[u], b[v], acc[u][v]);
        }
        __syncthreads();
    }
    float *y = (float *)(UK ? p.k : p.v) + (size_t)blockIdx.z * p.cap_rows * N;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const bool odd = p.odd[m0 + 4 * ty + u];
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (j0 + 4 * tx + v < N)
                y[(size_t)(m0 + 4 * ty + u) * N + j0 + 4 * tx + v] = odd ? (UK ? CUDART_NAN_F : 0.f) : acc[u][v];
    }
}

constexpr int kPQ = 16;   // new tokens per CTA
constexpr int kPT = 32;   // cached tokens per step

// One head's attention of kPQ new tokens: scores with one lane per cached token, softmax
// statistics per row in log2 units, then P . V into per-thread accumulators (thread owns
// value dims tid + 256 c of every row).
template <typename T, int NC>
__global__ void __launch_bounds__(256) prefill_simt_kernel(PrefillParams p) {
    extern __shared__ float smem[];
    if ((int)blockIdx.x >= p.tile_off[p.B]) return;
    const int b = find_seq(p.tile_off, p.B, blockIdx.x);
    const int hl = blockIdx.y, h = p.h0 + hl;
    const int dn = p.dn, dR = p.s.dR, dqk = dn + dR, dv = p.s.dv, D = p.s.D(), H = p.s.H;
    const int n = p.cu_q[b + 1] - p.cu_q[b], i0 = ((int)blockIdx.x - p.tile_off[b]) * kPQ;
    const int rows_here = min(kPQ, n - i0);
    const size_t qrow0 = (size_t)p.cu_q[b] + i0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    T *out = (T *)p.out;
    if (p.bad[b]) {
        for (int e = tid; e < rows_here * dv; e += 256)
            out[((qrow0 + e / dv) * H + h) * dv + e % dv] = (T)CUDART_NAN_F;
        if (p.lse && tid < rows_here) p.lse[(qrow0 + tid) * H + h] = CUDART_NAN_F;
        return;
    }
    const int L = p.seq_lens[b];
    const int Dp = dqk + 1;
    float *sQ = smem;                     // [kPQ][dqk]
    float *sK = sQ + kPQ * dqk;           // [kPT][Dp]
    float *sP = sK + kPT * Dp;            // [kPQ][kPT]
    float *sA = sP + kPQ * kPT;           // [kPQ]
    float *sL = sA + kPQ, *sM = sL + kPQ;
    const T *q = (const T *)p.q;
    for (int e = tid; e < kPQ * dqk; e += 256) {
        const int rr = e / dqk, d = e % dqk;
        sQ[e] = rr < rows_here ? to_f32(q[((qrow0 + rr) * H + h) * dqk + d]) : 0.f;
    }
    const size_t row0 = (size_t)p.kv_off[b];
    const float *K = (const float *)p.k + ((size_t)hl * p.cap_rows + row0) * dn;
    const float *V = (const float *)p.v + ((size_t)hl * p.cap_rows + row0) * dv;
    const T *rope = (const T *)p.rows + row0 * D + p.s.r;
    const float c2 = p.scale * kLog2e;
    float m_run[2] = {-CUDART_INF_F, -CUDART_INF_F}, l_run[2] = {0.f, 0.f};
    float acc[kPQ][NC];
#pragma unroll
    for (int rr = 0; rr < kPQ; ++rr)
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[rr][c] = 0.f;
    const int t_end = L - n + i0 + rows_here;            // tokens the last row sees
    for (int t0 = 0; t0 < t_end; t0 += kPT) {
        __syncthreads();
        for (int e = tid; e < kPT * dqk; e += 256) {
            const int tt = e / dqk, d = e % dqk;
            float v = 0.f;
            if (t0 + tt < t_end) v = d < dn ? K[(size_t)(t0 + tt) * dn + d] : to_f32(rope[(size_t)(t0 + tt) * D + d - dn]);
            sK[tt * Dp + d] = v;
        }
        __syncthreads();
        const float *q0 = sQ + warp * dqk, *q1 = sQ + (warp + 8) * dqk, *kr = sK + lane * Dp;
        float sc[2] = {0.f, 0.f};
        for (int d = 0; d < dqk; ++d) {
            sc[0] = fmaf(q0[d], kr[d], sc[0]);
            sc[1] = fmaf(q1[d], kr[d], sc[1]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int rr = warp + 8 * j;
            const bool vis = rr < rows_here && t0 + lane <= L - n + i0 + rr;
            const float s2 = vis ? sc[j] * c2 : -CUDART_INF_F;
            const float m_new = fmaxf(m_run[j], warp_max(s2));
            // (a score of minus infinity weighs 0, also while there is no other: m_new is it too)
            const float pr = s2 != -CUDART_INF_F ? exp2f(s2 - m_new) : 0.f;
            const float alpha = m_new == -CUDART_INF_F ? 1.f : exp2f(m_run[j] - m_new);
            l_run[j] = l_run[j] * alpha + warp_sum(pr);
            m_run[j] = m_new;
            sP[rr * kPT + lane] = pr;
            if (lane == 0) sA[rr] = alpha;
        }
        __syncthreads();
#pragma unroll
        for (int rr = 0; rr < kPQ; ++rr) {
            const float a = sA[rr];
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[rr][c] *= a;
        }
        const int nt = min(kPT, t_end - t0);
        for (int tt = 0; tt < nt; ++tt) {
            float vv[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) vv[c] = tid + 256 * c < dv ? V[(size_t)(t0 + tt) * dv + tid + 256 * c] : 0.f;
#pragma unroll
            for (int rr = 0; rr < kPQ; ++rr) {
                const float pr = sP[rr * kPT + tt];
#pragma unroll
                for (int c = 0; c < NC; ++c) acc[rr][c] = fmaf(pr, vv[c], acc[rr][c]);
            }
        }
    }
    if (lane == 0)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            sL[warp + 8 * j] = l_run[j];
            sM[warp + 8 * j] = m_run[j];
        }
    __syncthreads();
#pragma unroll
    for (int rr = 0; rr < kPQ; ++rr) {
        if (rr >= rows_here) break;
        const float inv = 1.f / sL[rr];
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (tid + 256 * c < dv) out[((qrow0 + rr) * H + h) * dv + tid + 256 * c] = (T)(acc[rr][c] * inv);
    }
    if (p.lse && tid < rows_here) p.lse[(qrow0 + tid) * H + h] = (sM[tid] + log2f(sL[tid])) * kLn2;
}

static constexpr size_t prefill_smem(size_t dqk) {
    return sizeof(float) * (kPQ * dqk + kPT * (dqk + 1) + kPQ * kPT + 3 * kPQ);
}

template <typename T>
static cudaError_t prefill_simt_t(const PrefillParams &p, cudaStream_t st) {
    const unsigned mt = (unsigned)(p.cap_rows / 64);
    expand_simt_kernel<T, true><<<dim3(mt, (p.dn + 63) / 64, p.nh), 256, 0, st>>>(p);
    expand_simt_kernel<T, false><<<dim3(mt, (p.s.dv + 63) / 64, p.nh), 256, 0, st>>>(p);
    const size_t smem = prefill_smem(p.dn + p.s.dR);
    const dim3 grid((unsigned)(p.num_q / kPQ + p.B), p.nh);
    auto go = [&](void (*kern)(PrefillParams)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)prefill_smem(kMaxNope + kMaxRope));
        if (e != cudaSuccess) return e;
        kern<<<grid, 256, smem, st>>>(p);
        return cudaGetLastError();
    };
    if (p.s.dv <= 256) return go(prefill_simt_kernel<T, 1>);
    if (p.s.dv <= 512) return go(prefill_simt_kernel<T, 2>);
    return go(prefill_simt_kernel<T, 4>);
}

cudaError_t launch_prefill_simt(const PrefillParams &p, cudaStream_t st) {
    return p.s.kind == MLA_KV_FP32 ? prefill_simt_t<float>(p, st) : prefill_simt_t<__nv_bfloat16>(p, st);
}

}  // namespace mla
