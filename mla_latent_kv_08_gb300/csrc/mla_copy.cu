// Copies of cached rows, in the caches of many layers with one launch (mla_cache_copy).
//
// An entry (src, dst, first, rows) moves rows first .. first + rows - 1 of block src to the
// same rows of block dst. The rows of a block are contiguous in each of a cache's arrays, so
// that an entry is up to three contiguous pieces a layer. Memory bound: the bytes once in,
// once out. A CTA takes kPart bytes of an entry at a time, all of which it loads before it
// stores any: kUnroll 16-byte loads a thread. 200 whole blocks of the 8-bit cache in 24 layers (403 MB
// in and out): 63.1 us, 6.4 TB/s of the copy rate's 6.7 (array by array, with 8 CTAs an SM: 78 us;
// 8 KB a task: 93 us, 32 KB: 71 us); of bf16 rows (708 MB) 107.7 us, 6.6 TB/s; of fp32 ones (1416 MB)
// 212 us, 6.7 TB/s; of rotated 2-bit ones (197 MB) 34.5 us, 5.7 TB/s; with the rope key as codes too
// (133 MB) 26.4 us, 5.0 TB/s: its rows of 144 and 72 bytes go in 8-byte loads, since all loads are as wide
// as the narrowest array has them. 24 tails of 1 to 64 rows in 32 layers (61 MB): 11.9 us (13.3 where a
// bf16 row's one array goes the way of three); 8 in one layer: 1.7 us. An empty list costs 1 to 3 us,
// by the CTAs that its room asks for: 16 an SM at most (24 would copy 1 to 2 % faster).
#include "mla_internal.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr int kPart = kThreads * kUnroll * 16;       // bytes of a CTA's task, at most

// U: the type of a load, which divides every row's bytes. ARRAYS: of a cache, 1 or 3.
template <typename U, int ARRAYS>
__global__ void __launch_bounds__(kThreads) copy_kernel(const __grid_constant__ CopyParams p, int part_rows, unsigned parts) {
    pdl_wait();
    pdl_trigger();
    const int layer = blockIdx.y, tid = threadIdx.x;
    const unsigned n = max(0, min(*p.num_copies, p.max_copies));
    const int u0 = p.row_bytes[0] / sizeof(U), u1 = p.row_bytes[1] / sizeof(U), u2 = p.row_bytes[2] / sizeof(U);
    U *const p0 = (U *)p.plane[layer][0], *const p1 = (U *)p.plane[layer][1], *const p2 = (U *)p.plane[layer][2];
    // a task is a part of an entry; all of them may be more than 2^32
    const unsigned step = gridDim.x / parts, step_part = gridDim.x % parts;
    unsigned entry = blockIdx.x / parts, part = blockIdx.x % parts;
    int4 next = entry < n ? p.copies[entry] : make_int4(0, 0, 0, 0);
    while (entry < n) {
        const int4 c = next;
        const int at = part * part_rows;
        entry += step;
        part += step_part;
        if (part >= parts) {
            part -= parts;
            ++entry;
        }
        if (entry < n) next = p.copies[entry];
        const bool ok = c.x >= 0 && c.x < p.num_blocks && c.y >= 0 && c.y < p.num_blocks && c.z >= 0 && c.w >= 0 &&
                        c.z <= p.bs && c.w <= p.bs - c.z;
        if (!ok) {
            if (tid == 0) raise_flag(p.status, FLAG_BAD_BLOCK);
            continue;
        }
        const int rows = min(part_rows, c.w - at);
        if (rows <= 0 || c.x == c.y) continue;
        // the rows are contiguous in each array; the arrays' pieces are numbered one behind the other
        const size_t from = (size_t)c.x * p.bs + c.z + at, to = (size_t)c.y * p.bs + c.z + at;
        const int m0 = rows * u0, m1 = m0 + rows * u1, m = ARRAYS == 1 ? m0 : m1 + rows * u2;
        const U *const s0 = p0 + from * u0, *const s1 = p1 + from * u1, *const s2 = p2 + from * u2;
        U *const d0 = p0 + to * u0, *const d1 = p1 + to * u1, *const d2 = p2 + to * u2;
        for (int i0 = tid; i0 < m; i0 += kUnroll * kThreads) {
            U v[kUnroll];
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) {
                const int i = i0 + j * kThreads;
                if (i < m) v[j] = ARRAYS == 1 || i < m0 ? s0[i] : i < m1 ? s1[i - m0] : s2[i - m1];
            }
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) {
                const int i = i0 + j * kThreads;
                if (i < m) *(ARRAYS == 1 || i < m0 ? d0 + i : i < m1 ? d1 + (i - m0) : d2 + (i - m1)) = v[j];
            }
        }
    }
}

template <typename U>
cudaError_t launch(const CopyParams &p, dim3 grid, int part_rows, unsigned parts, cudaStream_t st) {
    return launch_pdl(p.row_bytes[1] ? copy_kernel<U, 3> : copy_kernel<U, 1>, grid, dim3(kThreads), 0, st, p, part_rows, parts);
}

}  // namespace

cudaError_t launch_copy(const CopyParams &p, int32_t layers, cudaStream_t st) {
    int row = 0, bits = 16;
    for (int k = 0; k < 3; ++k) {
        row += p.row_bytes[k];
        bits |= p.row_bytes[k];
    }
    const int part_rows = row >= kPart ? 1 : kPart / row < p.bs ? kPart / row : p.bs;
    const unsigned parts = ((unsigned)p.bs + part_rows - 1) / part_rows;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int64_t tasks = (int64_t)p.max_copies * parts, most = (16ll * sms + layers - 1) / layers;
    const dim3 grid((unsigned)(tasks < most ? tasks : most), (unsigned)layers);
    switch (bits & -bits) {                  // rows begin at multiples of it in every array
        case 16: return launch<uint4>(p, grid, part_rows, parts, st);
        case 8: return launch<uint2>(p, grid, part_rows, parts, st);
        case 4: return launch<uint32_t>(p, grid, part_rows, parts, st);
        case 2: return launch<uint16_t>(p, grid, part_rows, parts, st);
        default: return launch<uint8_t>(p, grid, part_rows, parts, st);
    }
}

}  // namespace mla
