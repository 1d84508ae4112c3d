// Copies of cached rows, in the caches of many layers with one launch (mla_cache_copy).
//
// An entry (src, dst, first, rows) moves rows first .. first + rows - 1 of block src to the
// same rows of block dst. The rows of a block are contiguous in each of a cache's arrays, so
// that an entry is up to three contiguous pieces a layer. Memory bound: the bytes once in,
// once out. A CTA takes kPart bytes of an entry at a time.
#include "mla_internal.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kPart = 16384;                 // bytes of a CTA's task, about

// U: the type of a load, which divides every row's bytes.
template <typename U>
__global__ void __launch_bounds__(kThreads) copy_kernel(const __grid_constant__ CopyParams p, int part_rows, int parts) {
    constexpr int kSize = sizeof(U);
    pdl_wait();
    pdl_trigger();
    const int layer = blockIdx.y;
    const int n = max(0, min(*p.num_copies, p.max_copies));
    for (int task = blockIdx.x; task < n * parts; task += gridDim.x) {
        const int e = task / parts, at = (task - e * parts) * part_rows;
        const int4 c = p.copies[e];
        const bool ok = c.x >= 0 && c.x < p.num_blocks && c.y >= 0 && c.y < p.num_blocks && c.z >= 0 && c.w >= 0 &&
                        c.z <= p.bs && c.w <= p.bs - c.z;
        if (!ok) {
            if (threadIdx.x == 0) raise_flag(p.status, FLAG_BAD_BLOCK);
            continue;
        }
        const int rows = min(part_rows, c.w - at);
        if (rows <= 0 || c.x == c.y) continue;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int rb = p.row_bytes[k];
            if (rb == 0) continue;
            const size_t from = ((size_t)c.x * p.bs + c.z + at) * rb, to = ((size_t)c.y * p.bs + c.z + at) * rb;
            const U *src = (const U *)(p.plane[layer][k] + from);
            U *dst = (U *)(p.plane[layer][k] + to);
            const int m = rows * (rb / kSize);
            for (int i = threadIdx.x; i < m; i += 4 * kThreads) {
                U v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (i + j * kThreads < m) v[j] = src[i + j * kThreads];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (i + j * kThreads < m) dst[i + j * kThreads] = v[j];
            }
        }
    }
}

}  // namespace

cudaError_t launch_copy(const CopyParams &p, int32_t layers, cudaStream_t st) {
    int row = 0, bits = 16;
    for (int k = 0; k < 3; ++k) {
        row += p.row_bytes[k];
        bits |= p.row_bytes[k];
    }
    const int part_rows = row >= kPart ? 1 : kPart / row < p.bs ? kPart / row : p.bs;
    const int parts = (p.bs + part_rows - 1) / part_rows;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int64_t tasks = (int64_t)p.max_copies * parts, most = (8ll * sms + layers - 1) / layers;
    const dim3 grid((unsigned)(tasks < most ? tasks : most), (unsigned)layers);
    switch (bits & -bits) {                  // rows begin at multiples of it in every array
        case 16: return launch_pdl(copy_kernel<uint4>, grid, dim3(kThreads), 0, st, p, part_rows, parts);
        case 8: return launch_pdl(copy_kernel<uint2>, grid, dim3(kThreads), 0, st, p, part_rows, parts);
        case 4: return launch_pdl(copy_kernel<uint32_t>, grid, dim3(kThreads), 0, st, p, part_rows, parts);
        case 2: return launch_pdl(copy_kernel<uint16_t>, grid, dim3(kThreads), 0, st, p, part_rows, parts);
        default: return launch_pdl(copy_kernel<uint8_t>, grid, dim3(kThreads), 0, st, p, part_rows, parts);
    }
}

}  // namespace mla
