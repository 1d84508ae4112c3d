// Reading the paged cache back as dense rows, for every cache kind.
//
// bf16 (BF16, MXFP8) or fp32 (FP32, INT2) rows of r + d_R values. Memory bound: a token's
// stored bytes in, its row out (MXFP8 of the DeepSeek-V3 shape: 656 in, 1152 out). The lanes
// of a warp look the tokens of its eight rows up side by side (a chain of dependent loads
// that a warp a row would pay for each), then the warp moves two rows at a time. 133k MXFP8
// tokens: 43.9 us, 5.5 TB/s of the copy rate's 6.8 (a warp a row: 55 us; without the look for
// codes that are not a number 42.7); up to 4096 rows a warp a row fills more SMs (1000 tokens:
// 2.7 us).
#include "mla_internal.cuh"
#include "mla_mx.cuh"

#include <math_constants.h>

namespace mla {

enum : long long { kSkip = -1, kBadRow = -2, kZeroRow = -3 };

// Whether a 16-byte piece has an infinity or a NaN among its values.
template <int EL>
__device__ __forceinline__ bool not_finite(const uint4 &u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    bool b = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        b |= EL == 4 ? (w[i] & 0x7f800000u) == 0x7f800000u
                     : (w[i] & 0x7f800000u) == 0x7f800000u || (w[i] & 0x7f80u) == 0x7f80u;
    return b;
}

// Rows n[0..N) from token rows tok[0..N) (kSkip: none), by one warp.
template <int KIND, int N>
__device__ __forceinline__ void write_rows(const ReadParams &p, const long long (&tok)[N], size_t n0) {
    const int lane = threadIdx.x & 31;
    const int r = p.s.r, dR = p.s.dR, D = r + dR;
    if (KIND == MLA_KV_BF16 || KIND == MLA_KV_FP32) {
        constexpr int kEl = KIND == MLA_KV_BF16 ? 2 : 4;
        const int nv = D * kEl / 16, nl = r * kEl / 16;
        uint32_t odd = 0;                              // bit i: this lane saw one in row i
        for (int v0 = 0; v0 < nv; v0 += 96) {
            uint4 u[N][3];
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    const int v = v0 + 32 * k + lane;
                    if (tok[i] >= 0 && v < nv)
                        u[i][k] = ((const uint4 *)((const uint8_t *)p.latent + (size_t)tok[i] * p.s.E() * kEl))[v];
                }
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    const int v = v0 + 32 * k + lane;
                    if (tok[i] >= 0 && v < nv) ((uint4 *)((uint8_t *)p.rows + (n0 + i) * D * kEl))[v] = u[i][k];
                    if (p.odd && tok[i] >= 0 && v < nl) odd |= (uint32_t)not_finite<kEl>(u[i][k]) << i;
                }
        }
        if (p.odd)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const bool any = __any_sync(0xffffffffu, odd >> i & 1u);
                if (lane == 0 && tok[i] >= 0) p.odd[n0 + i] = any;
            }
    } else if (KIND == MLA_KV_MXFP8) {
        const int nv = r / 8, rv = dR / 8;             // eight values at a time
        uint32_t odd = 0;                              // bit i: this lane saw one in row i
        for (int v0 = 0; v0 < nv; v0 += 64) {
            uint2 c[N][2];
            uint32_t sb[N][2];
            uint4 rope[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int v = v0 + 32 * k + lane;
                    if (tok[i] >= 0 && v < nv) {
                        c[i][k] = ((const uint2 *)(p.codes + (size_t)tok[i] * r))[v];
                        sb[i][k] = p.mx_scale[(size_t)tok[i] * (r / kMxGroup) + v / 4];
                    }
                }
                if (v0 == 0 && tok[i] >= 0 && lane < rv) rope[i] = ((const uint4 *)(p.rope + (size_t)tok[i] * dR))[lane];
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                uint4 *dst = (uint4 *)((__nv_bfloat16 *)p.rows + (n0 + i) * D);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int v = v0 + 32 * k + lane;
                    if (tok[i] >= 0 && v < nv) {
                        dst[v] = mx_expand8(c[i][k], mx_scale_bf162(sb[i][k]));
                        odd |= (uint32_t)(sb[i][k] == 255u || mx_any_nan(c[i][k])) << i;
                    }
                }
                if (v0 == 0 && tok[i] >= 0 && lane < rv) dst[nv + lane] = rope[i];      // d_R <= 128: 16 lanes
            }
        }
        if (p.odd)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const bool any = __any_sync(0xffffffffu, odd >> i & 1u);
                if (lane == 0 && tok[i] >= 0) p.odd[n0 + i] = any;
            }
    } else {
#pragma unroll 1
        for (int i = 0; i < N; ++i) {
            if (tok[i] < 0) continue;
            float *dst = (float *)p.rows + (n0 + i) * D;
            const int QD = p.s.QD(), gs = p.s.gs, ng = QD / gs;
            for (int k = lane; k < QD / 4; k += 32) {
                const unsigned byte = p.codes[(size_t)tok[i] * (QD / 4) + k];
                const __half *sz = p.scale_zero + ((size_t)tok[i] * ng + 4 * k / gs) * 2;
                const float sc = __half2float(sz[0]), zr = __half2float(sz[1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) dst[4 * k + e] = __fmaf_rn((float)((byte >> (2 * e)) & 3u), sc, zr);
            }
            if (QD == r)
                for (int d = lane; d < dR; d += 32) dst[r + d] = __bfloat162float(p.rope[(size_t)tok[i] * dR + d]);
        }
    }
}

// Every element of row n as `v` (0 or NaN).
template <int KIND>
__device__ __forceinline__ void fill_row(const ReadParams &p, size_t n, float v) {
    const int lane = threadIdx.x & 31, D = p.s.D();
    if (p.odd && lane == 0) p.odd[n] = 0;
    if (KIND == MLA_KV_BF16 || KIND == MLA_KV_MXFP8) {
        __nv_bfloat16 *dst = (__nv_bfloat16 *)p.rows + n * D;
        for (int d = lane; d < D; d += 32) dst[d] = __float2bfloat16_rn(v);
    } else {
        float *dst = (float *)p.rows + n * D;
        for (int d = lane; d < D; d += 32) dst[d] = v;
    }
}

// The token row of output row n, or what to do with it.
__device__ __forceinline__ long long find_token(const ReadParams &p, int n) {
    if (n >= p.num_rows || n >= p.cu_rows[p.B]) return kSkip;
    const int b = find_seq(p.cu_rows, p.B, n);
    const int t = n - p.cu_rows[b];
    if (t < 0) return kSkip;                                        // before the first sequence's rows
    if (p.lens && t >= p.lens[b]) return kZeroRow;                  // padding of the prefill's rows
    const long long pos = (p.start_pos ? (long long)p.start_pos[b] : 0ll) + t;
    int blk = -1, lb = 0;
    if (pos >= 0 && pos <= INT32_MAX) {
        lb = (int)((uint32_t)pos / (uint32_t)p.s.bs);
        if (lb < p.max_blocks) blk = p.block_table[(size_t)b * p.max_blocks + lb];
    }
    if (blk < 0 || blk >= p.s.num_blocks) {
        raise_flag(p.status, FLAG_BAD_BLOCK);
        if (p.bad) p.bad[b] = 1;
        return p.lens ? kZeroRow : kBadRow;
    }
    return (long long)blk * p.s.bs + (pos - (long long)lb * p.s.bs);
}

template <int KIND, int N>              // N rows a warp, two at a time
__global__ void __launch_bounds__(256, KIND == MLA_KV_MXFP8 || KIND == MLA_KV_BF16 ? 5 : 4) read_kernel(ReadParams p) {
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    const long long n0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * N;
    if (n0 >= p.num_rows) return;
    const long long mine = lane < N ? find_token(p, (int)min(n0 + lane, (long long)INT32_MAX)) : kSkip;
    constexpr int M = N > 1 ? 2 : 1;
#pragma unroll 1
    for (int i = 0; i < N; i += M) {
        long long tok[M];
#pragma unroll
        for (int k = 0; k < M; ++k) tok[k] = __shfl_sync(0xffffffffu, mine, i + k);
        write_rows<KIND, M>(p, tok, (size_t)(n0 + i));
#pragma unroll
        for (int k = 0; k < M; ++k)
            if (tok[k] == kBadRow || tok[k] == kZeroRow)
                fill_row<KIND>(p, (size_t)(n0 + i + k), tok[k] == kBadRow ? CUDART_NAN_F : 0.f);
    }
}

template <int KIND>
static cudaError_t launch_kind(const ReadParams &p, cudaStream_t st) {
    // a warp a row while that leaves SMs free, else eight rows a warp
    const bool many = p.num_rows > 4096;
    const auto kern = many ? read_kernel<KIND, 8> : read_kernel<KIND, 1>;
    const dim3 grid((unsigned)(many ? (p.num_rows + 63ll) / 64 : (p.num_rows + 7ll) / 8));
    if (p.lens) return launch_pdl(kern, grid, dim3(256), 0, st, p);      // behind the prefill's plan
    kern<<<grid, 256, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_read(const ReadParams &p, cudaStream_t st) {
    if (p.num_rows == 0) return cudaSuccess;
    switch (p.s.kind) {
        case MLA_KV_BF16: return launch_kind<MLA_KV_BF16>(p, st);
        case MLA_KV_FP32: return launch_kind<MLA_KV_FP32>(p, st);
        case MLA_KV_MXFP8: return launch_kind<MLA_KV_MXFP8>(p, st);
        default: return launch_kind<MLA_KV_INT2_ROT>(p, st);
    }
}

}  // namespace mla
