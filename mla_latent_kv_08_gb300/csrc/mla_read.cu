// Reading the paged cache back as dense rows, for every cache kind: one warp a row.
//
// bf16 (BF16, MXFP8) or fp32 (FP32, INT2) rows of r + d_R values. Memory bound: a token's
// stored bytes in, its row out (MXFP8 of the DeepSeek-V3 shape: 656 in, 1152 out).
#include "mla_internal.cuh"
#include "mla_mx.cuh"

#include <math_constants.h>

namespace mla {

template <int KIND>
__device__ __forceinline__ void write_row(const ReadParams &p, long long tok, size_t n) {
    const int lane = threadIdx.x & 31;
    const int r = p.s.r, dR = p.s.dR, D = r + dR;
    if (KIND == MLA_KV_BF16 || KIND == MLA_KV_FP32) {
        constexpr int kEl = KIND == MLA_KV_BF16 ? 2 : 4;
        const uint4 *src = (const uint4 *)((const uint8_t *)p.latent + (size_t)tok * p.s.E() * kEl);
        uint4 *dst = (uint4 *)((uint8_t *)p.rows + n * D * kEl);
        for (int v = lane; v < D * kEl / 16; v += 32) dst[v] = src[v];
    } else if (KIND == MLA_KV_MXFP8) {
        uint4 *dst = (uint4 *)((__nv_bfloat16 *)p.rows + n * D);
        const uint4 *codes = (const uint4 *)(p.codes + (size_t)tok * r);
        const uint8_t *scales = p.mx_scale + (size_t)tok * (r / kMxGroup);
        for (int v = lane; v < r / 16; v += 32) {
            const uint4 c = codes[v];
            uint4 o0, o1;
            mx_expand16(c, kMx2p120, mx_scale_bf162(scales[v >> 1]), o0, o1);
            dst[2 * v] = o0;
            dst[2 * v + 1] = o1;
        }
        const uint4 *rope = (const uint4 *)(p.rope + (size_t)tok * dR);
        for (int v = lane; v < dR / 8; v += 32) dst[r / 8 + v] = rope[v];
    } else {
        float *dst = (float *)p.rows + n * D;
        const int QD = p.s.QD(), gs = p.s.gs, ng = QD / gs;
        for (int k = lane; k < QD / 4; k += 32) {
            const unsigned byte = p.codes[(size_t)tok * (QD / 4) + k];
            const __half *sz = p.scale_zero + ((size_t)tok * ng + 4 * k / gs) * 2;
            const float sc = __half2float(sz[0]), zr = __half2float(sz[1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[4 * k + e] = __fmaf_rn((float)((byte >> (2 * e)) & 3u), sc, zr);
        }
        if (QD == r)
            for (int d = lane; d < dR; d += 32) dst[r + d] = __bfloat162float(p.rope[(size_t)tok * dR + d]);
    }
}

// Every element of row n as `v` (0 or NaN).
template <int KIND>
__device__ __forceinline__ void fill_row(const ReadParams &p, size_t n, float v) {
    const int lane = threadIdx.x & 31, D = p.s.D();
    if (KIND == MLA_KV_BF16 || KIND == MLA_KV_MXFP8) {
        __nv_bfloat16 *dst = (__nv_bfloat16 *)p.rows + n * D;
        for (int d = lane; d < D; d += 32) dst[d] = __float2bfloat16_rn(v);
    } else {
        float *dst = (float *)p.rows + n * D;
        for (int d = lane; d < D; d += 32) dst[d] = v;
    }
}

template <int KIND>
__global__ void __launch_bounds__(256) read_kernel(ReadParams p) {
    const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (n >= p.num_rows || n >= p.cu_rows[p.B]) return;
    const int b = find_seq(p.cu_rows, p.B, n);
    const int t = n - p.cu_rows[b];
    if (t < 0) return;                                  // before the first sequence's rows
    if (p.lens && t >= p.lens[b]) {                     // padding of the prefill's rows
        fill_row<KIND>(p, n, 0.f);
        return;
    }
    const long long pos = (p.start_pos ? (long long)p.start_pos[b] : 0ll) + t;
    const long long lb = pos / p.s.bs;
    int blk = -1;
    if (pos >= 0 && lb < p.max_blocks) blk = p.block_table[(size_t)b * p.max_blocks + lb];
    if (blk < 0 || blk >= p.s.num_blocks) {
        if ((threadIdx.x & 31) == 0) {
            raise_flag(p.status, FLAG_BAD_BLOCK);
            if (p.bad) p.bad[b] = 1;
        }
        fill_row<KIND>(p, n, p.lens ? 0.f : CUDART_NAN_F);
        return;
    }
    write_row<KIND>(p, (long long)blk * p.s.bs + pos % p.s.bs, n);
}

cudaError_t launch_read(const ReadParams &p, cudaStream_t st) {
    if (p.num_rows == 0) return cudaSuccess;
    const dim3 grid((unsigned)((p.num_rows + 7ll) / 8));
    switch (p.s.kind) {
        case MLA_KV_BF16: read_kernel<MLA_KV_BF16><<<grid, 256, 0, st>>>(p); break;
        case MLA_KV_FP32: read_kernel<MLA_KV_FP32><<<grid, 256, 0, st>>>(p); break;
        case MLA_KV_MXFP8: read_kernel<MLA_KV_MXFP8><<<grid, 256, 0, st>>>(p); break;
        default: read_kernel<MLA_KV_INT2_ROT><<<grid, 256, 0, st>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace mla
