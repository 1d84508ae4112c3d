// The pool's books: which blocks sequences hold, and which are free (mla_pool_resize,
// mla_pool_fork, mla_pool_compact).
//
// A block is free if its count is 0. Free blocks are taken lowest first, in the order of the
// places that need one: prefix sums over the places and over the counts give every place its
// block, so that nothing depends on the order in which threads run. One cluster of CTAs, in
// phases with a cluster barrier between them: (1) what each sequence needs, what is free, and
// whether anything is wrong; (2) nothing at all if so; else blocks are handed out; (3) others
// are given back. Blocks that a call gives back are not handed out by it.
//
// A warp counts a contiguous part of the counts, 128 at a time. Lists of table entries are
// walked in pieces of kPiece entries, a warp a piece.
#include "mla_internal.cuh"

#include <cooperative_groups.h>

namespace cg = cooperative_groups;

namespace mla {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kPiece = 256;                  // table entries, 8 a lane

struct Shared {
    int scan[33];
    long long scan2[33];
    int warp[kWarps];                        // this CTA's warps: blocks counted
    int count, flags, freed;
};

// Sums of the CTAs' counts: before this one, all; and every CTA's flags.
struct Totals {
    int before, all, flags;
};
__device__ __forceinline__ Totals totals(const cg::cluster_group &cl, Shared &sh) {
    Totals t = {0, 0, 0};
    for (unsigned c = 0; c < cl.num_blocks(); ++c) {
        const Shared *o = cl.map_shared_rank(&sh, c);
        if (c == cl.block_rank()) t.before = t.all;
        t.all += o->count;
        t.flags |= o->flags;
    }
    return t;
}

// The part of the counts that warp w of all counts, in steps of 128.
__device__ __forceinline__ int part_begin(int N, int64_t w, int64_t warps) {
    const int64_t steps = (N + 127ll) / 128;
    return (int)min((int64_t)N, steps * w / warps * 128);
}

// Whether blocks i0 + lane + 32 k below `end`, k = 0 .. 3, are free.
struct Free4 {
    bool v[4];
};
__device__ __forceinline__ Free4 free4(const int32_t *ref, int i0, int end) {
    Free4 f;
    int c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int i = i0 + 32 * k + (threadIdx.x & 31);
        c[k] = i < end ? ref[i] : 1;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) f.v[k] = c[k] == 0;
    return f;
}

// Counts the free blocks of every warp's part into sh.warp and sh.count. The caller
// synchronises the block, then the cluster.
__device__ __forceinline__ void count_free(const PoolParams &p, Shared &sh, int64_t w, int64_t warps) {
    const int lane = threadIdx.x & 31, lo = part_begin(p.N, w, warps), hi = part_begin(p.N, w + 1, warps);
    int n = 0;
    for (int i0 = lo; i0 < hi; i0 += 128) {
        const Free4 f = free4(p.ref, i0, hi);
        n += f.v[0] + f.v[1] + f.v[2] + f.v[3];
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) {
        sh.warp[threadIdx.x >> 5] = n;
        if (n) atomicAdd(&sh.count, n);
    }
}

// give(rank, block) for each free block of rank below `need`, lowest first.
template <typename F>
__device__ __forceinline__ void hand_out(const PoolParams &p, const Shared &sh, int before, int need, int64_t w,
                                         int64_t warps, F give) {
    const int lane = threadIdx.x & 31, lo = part_begin(p.N, w, warps), hi = part_begin(p.N, w + 1, warps);
    int rank = before;
    for (int i = 0; i < (int)(threadIdx.x >> 5); ++i) rank += sh.warp[i];
    const uint32_t lower = (1u << lane) - 1;
    for (int i0 = lo; i0 < hi && rank < need; i0 += 128) {
        const Free4 f = free4(p.ref, i0, hi);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t m = __ballot_sync(0xffffffffu, f.v[k]);
            const int r = rank + __popc(m & lower);
            if (f.v[k] && r < need) give(r, i0 + 32 * k + lane);
            rank += __popc(m);
        }
    }
}

// f(list, entry) for the entries of lists whose pieces `pieces` counts: list b has the entries
// begin(b) .. end(b) - 1. All warps of the cluster take part.
template <typename R, typename F>
__device__ __forceinline__ void walk(const int *pieces, int lists, int64_t w, int64_t warps, R range, F f) {
    const int lane = threadIdx.x & 31, total = pieces[lists];
    for (int64_t c = w; c < total; c += warps) {
        const int b = find_seq(pieces, lists, (int)c);
        const int2 r = range(b);
        const int first = r.x + ((int)c - pieces[b]) * kPiece + lane;
#pragma unroll
        for (int k = 0; k < kPiece / 32; ++k)
            if (first + 32 * k < r.y) f(b, first + 32 * k);
    }
}

__device__ __forceinline__ int ceil_div(int a, int b) { return (int)(((unsigned)a + (unsigned)b - 1u) / (unsigned)b); }

// ---- resize -----------------------------------------------------------------

// What a sequence is to give and take: it holds `held` blocks and shall hold `wanted`; a cut
// inside a block that others hold too needs a block of its own (`old`: that block, else -1).
struct Change {
    int held, wanted, old, flags;
    __device__ __forceinline__ int takes() const { return (wanted > held ? wanted - held : 0) + (old >= 0); }
};
__device__ __forceinline__ Change change_of(const PoolParams &p, int b) {
    const int len = p.lens[b], to = p.new_lens[b];
    Change c = {0, 0, -1, 0};
    if (len < 0 || len > p.cap || to < 0 || to > p.cap) {
        c.flags = FLAG_BAD_LENGTH;
        return c;
    }
    c.held = ceil_div(len, p.bs);
    c.wanted = ceil_div(to, p.bs);
    if (to < len && to % p.bs) {
        const int t = p.table[(size_t)b * p.W + c.wanted - 1];
        if (t < 0 || t >= p.N) c.flags = FLAG_BAD_BLOCK;
        else if (p.ref[t] > 1) c.old = t;
    }
    return c;
}

__global__ void __launch_bounds__(kThreads) resize_kernel(const PoolParams p) {
    extern __shared__ int dyn[];
    __shared__ Shared sh;
    int *s_takes = dyn, *s_pieces = dyn + p.S + 1, *s_split = s_pieces + p.S + 1;      // [S + 1] each
    const cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x;
    const int64_t w = (int64_t)cl.block_rank() * kWarps + (tid >> 5), warps = (int64_t)cl.num_blocks() * kWarps;
    pdl_wait();
    pdl_trigger();
    if (tid == 0) sh.count = sh.flags = sh.freed = 0;
    __syncthreads();
    // every CTA: what each sequence takes, the pieces of what it gives back, whether its last
    // block is replaced
    int takes = 0, pieces = 0, splits = 0, flags = 0;
    for (int b0 = 0; b0 < p.S; b0 += kThreads) {
        const int b = b0 + tid;
        Change c = {0, 0, -1, 0};
        if (b < p.S) c = change_of(p, b);
        flags |= c.flags;
        const int back = c.held > c.wanted ? ceil_div(c.held - c.wanted, kPiece) : 0;
        long long all2;
        const long long two = block_exclusive_scan((long long)c.takes() << 32 | back, sh.scan2, all2);
        int all;
        const int one = block_exclusive_scan((int)(c.old >= 0), sh.scan, all);
        if (b < p.S) {
            s_takes[b] = takes + (int)(two >> 32);
            s_pieces[b] = pieces + (int)(two & 0xffffffff);
            s_split[b] = splits + one;
        }
        takes += (int)(all2 >> 32);
        pieces += (int)(all2 & 0xffffffff);
        splits += all;
    }
    if (tid == 0) {
        s_takes[p.S] = takes;
        s_pieces[p.S] = pieces;
        s_split[p.S] = splits;
    }
    __syncthreads();
    const auto given = [&](int b) { return make_int2(ceil_div(p.new_lens[b], p.bs), ceil_div(p.lens[b], p.bs)); };
    if (!__syncthreads_or(flags))            // lengths are fine: so are the ranges
        walk(s_pieces, p.S, w, warps, given, [&](int b, int j) {
            const int t = p.table[(size_t)b * p.W + j];
            if (t < 0 || t >= p.N) flags |= FLAG_BAD_BLOCK;
        });
    count_free(p, sh, w, warps);
    if (flags) atomicOr(&sh.flags, flags);
    __syncthreads();
    cl.sync();
    Totals t = totals(cl, sh);
    if (!t.flags && takes > t.all) t.flags = FLAG_FULL;
    if (t.flags) {                           // nothing is changed
        if (cl.block_rank() == 0 && tid == 0) {
            raise_flag(p.status, t.flags);
            *p.num_copies = 0;
            if (p.left) *p.left = t.all;
        }
        cl.sync();
        return;
    }
    hand_out(p, sh, t.before, takes, w, warps, [&](int r, int block) {
        const int b = find_seq(s_takes, p.S, r);
        const int len = p.lens[b], to = p.new_lens[b], k = r - s_takes[b];
        int32_t *row = p.table + (size_t)b * p.W;
        if (to < len) {                      // the cut's own copy of a shared block
            const int j = ceil_div(to, p.bs) - 1;
            p.copies[s_split[b]] = make_int4(row[j], block, 0, to % p.bs);
            row[j] = block;
        } else {
            row[ceil_div(len, p.bs) + k] = block;
        }
        p.ref[block] = 1;
    });
    cl.sync();                               // all free blocks have been looked at
    int freed = 0;
    const auto give_back = [&](int block) { freed += atomicSub(&p.ref[block], 1) == 1; };
    walk(s_pieces, p.S, w, warps, given, [&](int b, int j) {
        int32_t *at = p.table + (size_t)b * p.W + j;
        give_back(*at);
        *at = -1;
    });
    for (int64_t i = (int64_t)cl.block_rank() * kThreads + tid; i < splits; i += (int64_t)cl.num_blocks() * kThreads)
        give_back(p.copies[i].x);
    freed = __reduce_add_sync(0xffffffffu, freed);
    if ((tid & 31) == 0 && freed) atomicAdd(&sh.freed, freed);
    cl.sync();                               // lengths have been read
    for (int64_t b = (int64_t)cl.block_rank() * kThreads + tid; b < p.S; b += (int64_t)cl.num_blocks() * kThreads)
        p.lens[b] = p.new_lens[b];
    if (cl.block_rank() == 0 && tid == 0) {
        *p.num_copies = splits;
        int left = t.all - takes;
        for (unsigned c = 0; c < cl.num_blocks(); ++c) left += cl.map_shared_rank(&sh, c)->freed;
        if (p.left) *p.left = left;
    }
    cl.sync();
}

// ---- fork -------------------------------------------------------------------

__global__ void __launch_bounds__(kThreads) fork_kernel(const PoolParams p) {
    extern __shared__ int dyn[];
    __shared__ Shared sh;
    int *s_takes = dyn, *s_pieces = dyn + p.n + 1, *s_len = s_pieces + p.n + 1;         // [n + 1] each
    uint32_t *s_child = (uint32_t *)(s_len + p.n + 1);                                   // a bit a sequence
    const cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x;
    const int64_t w = (int64_t)cl.block_rank() * kWarps + (tid >> 5), warps = (int64_t)cl.num_blocks() * kWarps;
    pdl_wait();
    pdl_trigger();
    if (tid == 0) sh.count = sh.flags = sh.freed = 0;
    for (int i = tid; i < (p.S + 31) / 32; i += kThreads) s_child[i] = 0;
    __syncthreads();
    int takes = 0, pieces = 0, flags = 0;
    for (int i0 = 0; i0 < p.n; i0 += kThreads) {
        const int i = i0 + tid;
        int len = 0;
        if (i < p.n) {
            const int a = p.parents[i], c = p.children[i];
            if (a < 0 || a >= p.S || c < 0 || c >= p.S) {
                flags |= FLAG_BAD_LENGTH;
            } else {
                const int most = p.lens[a];
                len = p.fork_lens ? p.fork_lens[i] : most;
                const uint32_t bit = 1u << (c & 31);
                // an empty sequence, and each but once
                if (most < 0 || most > p.cap || len < 0 || len > most || p.lens[c] != 0 || (atomicOr(&s_child[c / 32], bit) & bit)) {
                    flags |= FLAG_BAD_LENGTH;
                    len = 0;
                }
            }
        }
        long long all;
        const long long two = block_exclusive_scan(
            (long long)(len % p.bs != 0) << 32 | ceil_div(len / p.bs, kPiece), sh.scan2, all);
        if (i < p.n) {
            s_takes[i] = takes + (int)(two >> 32);
            s_pieces[i] = pieces + (int)(two & 0xffffffff);
            s_len[i] = len;
        }
        takes += (int)(all >> 32);
        pieces += (int)(all & 0xffffffff);
    }
    if (tid == 0) {
        s_takes[p.n] = takes;
        s_pieces[p.n] = pieces;
    }
    __syncthreads();
    const auto common = [&](int i) { return make_int2(0, s_len[i] / p.bs); };
    if (!__syncthreads_or(flags)) {
        walk(s_pieces, p.n, w, warps, common, [&](int i, int j) {
            const int t = p.table[(size_t)p.parents[i] * p.W + j];
            if (t < 0 || t >= p.N) flags |= FLAG_BAD_BLOCK;
        });
        for (int i = tid; i < p.n; i += kThreads)
            if (s_len[i] % p.bs) {
                const int t = p.table[(size_t)p.parents[i] * p.W + s_len[i] / p.bs];
                if (t < 0 || t >= p.N) flags |= FLAG_BAD_BLOCK;
            }
    }
    count_free(p, sh, w, warps);
    if (flags) atomicOr(&sh.flags, flags);
    __syncthreads();
    cl.sync();
    Totals t = totals(cl, sh);
    if (!t.flags && takes > t.all) t.flags = FLAG_FULL;
    if (t.flags) {                           // nothing is changed
        if (cl.block_rank() == 0 && tid == 0) {
            raise_flag(p.status, t.flags);
            *p.num_copies = 0;
            if (p.left) *p.left = t.all;
        }
        cl.sync();
        return;
    }
    hand_out(p, sh, t.before, takes, w, warps, [&](int r, int block) {
        const int i = find_seq(s_takes, p.n, r), j = s_len[i] / p.bs;
        p.copies[r] = make_int4(p.table[(size_t)p.parents[i] * p.W + j], block, 0, s_len[i] % p.bs);
        p.table[(size_t)p.children[i] * p.W + j] = block;
        p.ref[block] = 1;
    });
    walk(s_pieces, p.n, w, warps, common, [&](int i, int j) {
        const int block = p.table[(size_t)p.parents[i] * p.W + j];
        p.table[(size_t)p.children[i] * p.W + j] = block;
        atomicAdd(&p.ref[block], 1);         // of a block in use: no free one is mistaken for it
    });
    for (int64_t i = (int64_t)cl.block_rank() * kThreads + tid; i < p.n; i += (int64_t)cl.num_blocks() * kThreads)
        p.lens[p.children[i]] = s_len[i];
    if (cl.block_rank() == 0 && tid == 0) {
        *p.num_copies = takes;
        if (p.left) *p.left = t.all - takes;
    }
    cl.sync();                               // nobody's numbers are read any longer
}

// ---- compact ----------------------------------------------------------------

__global__ void __launch_bounds__(kThreads) compact_kernel(const PoolParams p) {
    extern __shared__ int dyn[];
    __shared__ Shared sh;
    int *s_pieces = dyn;                     // [S + 1]
    const cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t w = (int64_t)cl.block_rank() * kWarps + warp, warps = (int64_t)cl.num_blocks() * kWarps;
    pdl_wait();
    pdl_trigger();
    if (tid == 0) sh.count = sh.flags = 0;
    __syncthreads();
    int pieces = 0, flags = 0;
    for (int b0 = 0; b0 < p.S; b0 += kThreads) {
        const int b = b0 + tid;
        int len = b < p.S ? p.lens[b] : 0;
        if (len < 0 || len > p.cap) {
            flags |= FLAG_BAD_LENGTH;
            len = 0;
        }
        int all;
        const int one = block_exclusive_scan(ceil_div(ceil_div(len, p.bs), kPiece), sh.scan, all);
        if (b < p.S) s_pieces[b] = pieces + one;
        pieces += all;
    }
    if (tid == 0) s_pieces[p.S] = pieces;
    if (flags) atomicOr(&sh.flags, flags);
    count_free(p, sh, w, warps);
    __syncthreads();
    cl.sync();
    const Totals t = totals(cl, sh);
    const int live = p.N - t.all;
    if (t.flags) {
        if (cl.block_rank() == 0 && tid == 0) {
            raise_flag(p.status, t.flags);
            *p.num_copies = 0;
            if (p.left) *p.left = live;
        }
        cl.sync();
        return;
    }
    // free blocks below `live`: those of the warps before the one with id `live`, and some of
    // that one's own. There are as many used blocks from `live` on.
    int64_t wl = 0;
    for (int64_t a = 0, e = warps; a < e;) {             // the last warp that begins at or below `live`
        const int64_t m = (a + e) / 2;
        if (part_begin(p.N, m, warps) <= live) { wl = m; a = m + 1; } else e = m;
    }
    int holes = 0;
    for (int64_t i = lane; i < wl; i += 32) holes += cl.map_shared_rank(&sh, (unsigned)(i / kWarps))->warp[i % kWarps];
    for (int i = part_begin(p.N, wl, warps) + lane; i < live; i += 32) holes += p.ref[i] == 0;
    holes = __reduce_add_sync(0xffffffffu, holes);
    const int moves = min(holes, p.n);
    // the k-th used block from `live` on goes to the k-th free one below
    {
        const int lo = part_begin(p.N, w, warps), hi = part_begin(p.N, w + 1, warps);
        int rank = t.before;                 // free blocks before
        for (int i = 0; i < warp; ++i) rank += sh.warp[i];
        const uint32_t lower = (1u << lane) - 1;
        for (int i0 = lo; i0 < hi; i0 += 128) {
            const Free4 f = free4(p.ref, i0, hi);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t mask = __ballot_sync(0xffffffffu, f.v[k]);
                const int r = rank + __popc(mask & lower), i = i0 + 32 * k + lane;
                rank += __popc(mask);
                if (i >= hi) continue;
                if (i < live) {
                    if (f.v[k] && r < moves) p.copies[r].y = i;
                } else if (!f.v[k]) {
                    const int m = i - live - (r - holes);            // used blocks from `live` on before this one
                    if (m < moves) {
                        p.copies[m].x = i;
                        p.copies[m].z = 0;
                        p.copies[m].w = p.bs;
                    }
                }
            }
        }
    }
    cl.sync();
    // a moved block's count goes with it; where it was, where it went is noted for the tables
    const int64_t thread = (int64_t)cl.block_rank() * kThreads + tid, threads = (int64_t)cl.num_blocks() * kThreads;
    for (int64_t i = thread; i < moves; i += threads) {
        const int4 c = p.copies[i];
        p.ref[c.y] = p.ref[c.x];
        p.ref[c.x] = ~c.y;
    }
    cl.sync();
    const auto held = [&](int b) { return make_int2(0, ceil_div(p.lens[b], p.bs)); };
    walk(s_pieces, p.S, w, warps, held, [&](int b, int j) {
        int32_t *at = p.table + (size_t)b * p.W + j;
        const int block = *at;
        if (block < 0 || block >= p.N) {
            raise_flag(p.status, FLAG_BAD_BLOCK);        // left as it is
        } else if (block >= live) {
            const int to = ~p.ref[block];
            if (to >= 0) *at = to;
        }
    });
    cl.sync();
    for (int64_t i = thread; i < moves; i += threads) p.ref[p.copies[i].x] = 0;
    if (cl.block_rank() == 0 && tid == 0) {
        *p.num_copies = moves;
        if (p.left) *p.left = live;
    }
}

constexpr unsigned kCluster = 1;

cudaError_t launch(void (*kern)(PoolParams), const PoolParams &p, size_t smem, cudaStream_t st) {
    if (smem > 40960) {                      // with the static part, more than a launch may have without asking
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_pool_resize(const PoolParams &p, cudaStream_t st) {
    return launch(resize_kernel, p, 3 * sizeof(int) * ((size_t)p.S + 1), st);
}
cudaError_t launch_pool_fork(const PoolParams &p, cudaStream_t st) {
    return launch(fork_kernel, p, 3 * sizeof(int) * ((size_t)p.n + 1) + sizeof(uint32_t) * (((size_t)p.S + 31) / 32), st);
}
cudaError_t launch_pool_compact(const PoolParams &p, cudaStream_t st) {
    return launch(compact_kernel, p, sizeof(int) * ((size_t)p.S + 1), st);
}

}  // namespace mla
