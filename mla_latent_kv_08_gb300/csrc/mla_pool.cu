// The pool's books: which blocks sequences hold, and which are free (mla_pool_resize,
// mla_pool_fork, mla_pool_compact).
//
// A block is free if its count is 0. Free blocks are taken lowest first, in the order of the
// places that need one: prefix sums over the places and over the counts give every place its
// block, so that nothing depends on the order in which threads run. One cluster of CTAs, in
// phases with a cluster barrier between them: (1) what each sequence needs, what is free, and
// whether anything is wrong; (2) nothing at all if so, else blocks are handed out; (3) others
// are given back. Blocks that a call gives back are not handed out by it.
//
// A warp counts a contiguous part of the counts, 128 at a time; consecutive parts belong to
// different CTAs, so that all of them hand out the lowest free blocks. Lists of table entries are
// walked in pieces of kPiece entries, a warp a piece, whose loads are all in flight before the
// first is used.
//
// Small calls are bound by their chain of dependent steps, of about half a microsecond each (a
// load from L2 takes 0.4, a cluster's barrier 0.5 to 1): a step of 32 sequences takes 5.7 us, a fork of
// one 4.7, compaction of 500 blocks 4.9. Large ones by the scattered accesses that 16 SMs can issue: 512
// sequences that give back 100k entries of 290k blocks 19.7 us (with a step's free blocks looked
// up one by one 32, with entries loaded one by one 36), 200 forks of 230k entries 16.6 us, 300k
// entries that follow 70k moved blocks 27.7 us. Walking them in a second kernel on all SMs took 19.3,
// 13.7 and 24.3 us when this took 21.1, 17.6 and 28.9, in two or three launches, which a call outside a
// captured graph pays for on the host.
#include "mla_internal.cuh"

#include <cooperative_groups.h>

#include <utility>

namespace cg = cooperative_groups;

namespace mla {
namespace {

constexpr int kMaxThreads = 1024, kMaxWarps = kMaxThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kPiece = 256;                  // table entries (a number of them, less one, fits a byte)

// What every CTA finds for itself: the blocks that the call takes, whether it gives any back,
// what is wrong.
struct Found {
    int takes, back, flags;
};

struct Shared {
    Found all[kMaxCluster];                  // of every CTA of the cluster
    int free[kMaxCluster * kMaxWarps];       // free blocks of every warp's part
    int2 scan[kMaxWarps];
    int scan_two[kMaxWarps];
    int warp[kMaxWarps];                     // this CTA's warps: free blocks of their parts
    int ids[kMaxWarps][128];                 // a step's free blocks
    int flags;
};

// Free blocks before this warp's part, all of them; every CTA's flags.
struct Totals {
    int before, all, flags;
};
// Every CTA tells every other, and waits for them. `here`: the cluster's arrival at the
// kernel's start, without which a CTA's shared memory may not be there yet. From here on
// all CTAs go the same way, whatever else: should they have found different things (books that
// another stream changes meanwhile), the call is refused.
__device__ __forceinline__ Totals exchange(const cg::cluster_group &cl, cg::cluster_group::arrival_token &here, Shared &sh,
                                           int w, int warps, int takes, int back) {
    const int tid = threadIdx.x, C = cl.num_blocks(), rank = cl.block_rank();
    cl.barrier_wait(std::move(here));
    __syncthreads();
    if (tid < warps) cl.map_shared_rank(&sh, tid % C)->free[tid / C * C + rank] = sh.warp[tid / C];
    if (tid < C) cl.map_shared_rank(&sh, tid)->all[rank] = Found{takes, back, sh.flags};
    cl.sync();
    Totals t = {0, 0, 0};
    for (int i = tid & 31; i < warps; i += 32) {
        const int n = sh.free[i];
        t.all += n;
        t.before += i < w ? n : 0;
    }
    t.all = __reduce_add_sync(0xffffffffu, t.all);
    t.before = __reduce_add_sync(0xffffffffu, t.before);
    for (int c = 0; c < C; ++c) {
        const Found &o = sh.all[c];
        t.flags |= o.flags;
        if (o.takes != sh.all[0].takes || o.back != sh.all[0].back) t.flags |= FLAG_BAD_LENGTH;
    }
    if (!t.flags && sh.all[0].takes > t.all) t.flags = FLAG_FULL;
    return t;
}

// Block-wide exclusive scan of three numbers a thread.
struct Three {
    int x, y, z;
};
__device__ __forceinline__ Three scan_three(Three v, Shared &sh, Three &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    Three in = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, in.x, o), y = __shfl_up_sync(0xffffffffu, in.y, o),
                  z = __shfl_up_sync(0xffffffffu, in.z, o);
        if (lane >= o) in.x += x, in.y += y, in.z += z;
    }
    __syncthreads();                         // the last scan's sums have been read
    if (lane == 31) {
        sh.scan[warp] = make_int2(in.x, in.y);
        sh.scan_two[warp] = in.z;
    }
    __syncthreads();
    // every warp adds the others' sums up for itself
    const int2 w = lane < warps ? sh.scan[lane] : make_int2(0, 0);
    const int wz = lane < warps ? sh.scan_two[lane] : 0;
    const bool before = lane < warp;
    const Three base = {__reduce_add_sync(0xffffffffu, before ? w.x : 0), __reduce_add_sync(0xffffffffu, before ? w.y : 0),
                        __reduce_add_sync(0xffffffffu, before ? wz : 0)};
    total = {__reduce_add_sync(0xffffffffu, w.x), __reduce_add_sync(0xffffffffu, w.y), __reduce_add_sync(0xffffffffu, wz)};
    return {base.x + in.x - v.x, base.y + in.y - v.y, base.z + in.z - v.z};
}

// The part of the counts that a warp counts, in steps of 128: `each` blocks a warp.
struct Parts {
    int64_t each;
    int N;
    __device__ __forceinline__ Parts(int N, int warps) : each((N + 127ll) / 128), N(N) {
        each = ((unsigned)each + (unsigned)warps - 1) / (unsigned)warps * 128ll;
    }
    __device__ __forceinline__ int begin(int w) const { return (int)min((int64_t)N, w * each); }
};

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

// Counts the free blocks of every warp's part into sh.warp.
__device__ __forceinline__ void count_free(const PoolParams &p, Shared &sh, const Parts &parts, int w) {
    const int lo = parts.begin(w), hi = parts.begin(w + 1);
    int n = 0;
#pragma unroll 4
    for (int i0 = lo; i0 < hi; i0 += 128) {
        const Free4 f = free4(p.ref, i0, hi);
        n += f.v[0] + f.v[1] + f.v[2] + f.v[3];
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if ((threadIdx.x & 31) == 0) sh.warp[threadIdx.x >> 5] = n;
}

// give(rank, block) for each free block of rank below `need`, lowest first. The free ones of
// a step are gathered first, so that whole warps look their places up.
__device__ __forceinline__ uint32_t lanes_below() { return (1u << (threadIdx.x & 31)) - 1; }
template <typename F>
__device__ __forceinline__ void hand_out(const PoolParams &p, Shared &sh, const Parts &parts, int w, int before, int need, F give) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lo = parts.begin(w), hi = parts.begin(w + 1);
    int rank = before;
    Free4 f = free4(p.ref, lo, rank < need ? hi : lo);
    for (int i0 = lo; i0 < hi && rank < need; i0 += 128) {
        const Free4 next = free4(p.ref, i0 + 128, hi);
        int n = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t m = __ballot_sync(0xffffffffu, f.v[k]);
            if (f.v[k]) sh.ids[warp][n + __popc(m & lanes_below())] = i0 + 32 * k + lane;
            n += __popc(m);
        }
        __syncwarp();
        for (int q = lane; q < min(n, need - rank); q += 32) give(rank + q, sh.ids[warp][q]);
        __syncwarp();
        rank += n;
        f = next;
    }
}

// f(list, first entry, values, how many) for the entries of lists whose pieces `pieces` counts:
// list b has the entries range(b).x .. range(b).y - 1 of the row row(b). A lane gets kLane
// entries of a piece, 32 apart. All warps of the cluster take part.
constexpr int kLane = kPiece / 32;
template <typename Range, typename Row, typename F>
__device__ __forceinline__ void walk(const int *pieces, int lists, int w, int warps, Range range, Row row, F f) {
    const int lane = threadIdx.x & 31, total = pieces[lists];
    for (int c = w; c < total; c += warps) {
        const int b = find_seq(pieces, lists, c);
        const int2 r = range(b);
        const int first = r.x + (c - pieces[b]) * kPiece + lane;
        const int32_t *from = row(b) + first;
        int v[kLane];
#pragma unroll
        for (int k = 0; k < kLane; ++k) v[k] = first + 32 * k < r.y ? from[32 * k] : 0;
        f(b, first, v, (r.y - first + 31) / 32);
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
__device__ __forceinline__ Change change_of(const PoolParams &p, int b, int len, int to) {
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

__global__ void __launch_bounds__(kMaxThreads, 1) resize_kernel(const PoolParams p) {
    extern __shared__ int dyn[];
    __shared__ Shared sh;
    int *s_takes = dyn, *s_pieces = dyn + p.S + 1;       // [S + 1] each
    int *s_place = s_pieces + p.S + 1;                   // [S] first entry that changes; ~(copy's number) for a cut's copy
    uint8_t *s_last = (uint8_t *)(s_place + p.S + 1);    // [S] entries of the last piece given back, less one
    const cg::cluster_group cl = cg::this_cluster();
    auto here = cl.barrier_arrive();
    const Parts parts(p.N, gridDim.x * blockDim.x / 32);
    const int tid = threadIdx.x, block = blockDim.x;
    const int thread = blockIdx.x * block + tid, threads = gridDim.x * block;       // of the cluster
    const int w = (tid >> 5) * gridDim.x + blockIdx.x, warps = threads >> 5;
    pdl_wait();
    pdl_trigger();
    if (tid == 0) sh.flags = 0;
    // every CTA: what each sequence takes, the pieces of what it gives back, whether its last
    // block is replaced
    Three sum = {0, 0, 0};
    int flags = 0, len = tid < p.S ? p.lens[tid] : 0, to = tid < p.S ? p.new_lens[tid] : 0;
    count_free(p, sh, parts, w);             // while these are on their way
    for (int b0 = 0; b0 < p.S; b0 += block) {
        const int b = b0 + tid;
        Change c = {0, 0, -1, 0};
        if (b < p.S) c = change_of(p, b, len, to);
        if (b + block < p.S) {
            len = p.lens[b + block];
            to = p.new_lens[b + block];
        }
        flags |= c.flags;
        Three all;
        const Three at = scan_three({c.takes(), c.held > c.wanted ? ceil_div(c.held - c.wanted, kPiece) : 0, c.old >= 0}, sh, all);
        if (b < p.S) {
            s_takes[b] = sum.x + at.x;
            s_pieces[b] = sum.y + at.y;
            s_place[b] = c.old >= 0 ? ~(sum.z + at.z) : min(c.held, c.wanted);
            s_last[b] = (uint8_t)(c.held - c.wanted - 1);
        }
        sum = {sum.x + all.x, sum.y + all.y, sum.z + all.z};
    }
    const int takes = sum.x, splits = sum.z;
    if (tid == 0) {
        s_takes[p.S] = takes;
        s_pieces[p.S] = sum.y;
    }
    const auto given = [&](int b) { return make_int2(ceil_div(p.new_lens[b], p.bs), ceil_div(p.lens[b], p.bs)); };
    const auto row = [&](int b) { return p.table + (size_t)b * p.W; };
    if (!__syncthreads_or(flags))            // lengths are fine: so are the ranges
        walk(s_pieces, p.S, w, warps, given, row, [&](int, int, const int (&v)[kLane], int n) {
#pragma unroll
            for (int k = 0; k < kLane; ++k)
                if (k < n && (v[k] < 0 || v[k] >= p.N)) flags |= FLAG_BAD_BLOCK;
        });
    if (flags) atomicOr(&sh.flags, flags);
    const bool back = sum.y > 0 || splits > 0;
    const Totals t = exchange(cl, here, sh, w, warps, takes, back);
    if (t.flags) {                           // nothing is changed
        if (thread == 0) {
            raise_flag(p.status, t.flags);
            *p.num_copies = 0;
            if (p.left) *p.left = t.all;
        }
        return;
    }
    hand_out(p, sh, parts, w, t.before, takes, [&](int r, int block) {
        const int b = find_seq(s_takes, p.S, r), place = s_place[b];
        int32_t *at = p.table + (size_t)b * p.W + place + (r - s_takes[b]);
        if (place < 0) {                     // the cut's own copy of a shared block
            const int to = p.new_lens[b];
            at = p.table + (size_t)b * p.W + ceil_div(to, p.bs) - 1;
            p.copies[~place] = make_int4(*at, block, 0, to % p.bs);
        }
        *at = block;
        p.ref[block] = 1;
    });
    for (int b = thread; b < p.S; b += threads) p.lens[b] = p.new_lens[b];
    if (thread == 0) {
        *p.num_copies = splits;
        if (p.left) *p.left = t.all - takes;
    }
    if (!back) return;
    cl.sync();                               // all free blocks have been looked at
    int freed = 0;
    // the entries of `given` once more: lengths are new ones now
    const auto rest = [&](int b) {
        const int first = s_place[b] >= 0 ? s_place[b] : ceil_div(p.new_lens[b], p.bs);
        return make_int2(first, first + (s_pieces[b + 1] - s_pieces[b] - 1) * kPiece + s_last[b] + 1);
    };
    walk(s_pieces, p.S, w, warps, rest, row, [&](int b, int j, const int (&v)[kLane], int n) {
        int32_t *at = p.table + (size_t)b * p.W + j;
        int old[kLane];
#pragma unroll
        for (int k = 0; k < kLane; ++k) {
            old[k] = 0;
            if (k < n && v[k] >= 0 && v[k] < p.N) {
                old[k] = atomicSub(&p.ref[v[k]], 1);
                at[32 * k] = -1;
            }
        }
#pragma unroll
        for (int k = 0; k < kLane; ++k) freed += old[k] == 1;
    });
    for (int i = thread; i < splits; i += threads) {
        const int old = p.copies[i].x;
        if (old >= 0 && old < p.N) freed += atomicSub(&p.ref[old], 1) == 1;
    }
    freed = __reduce_add_sync(0xffffffffu, freed);
    if (p.left && (tid & 31) == 0 && freed) atomicAdd(p.left, freed);
}

// ---- fork -------------------------------------------------------------------

__global__ void __launch_bounds__(kMaxThreads, 1) fork_kernel(const PoolParams p) {
    extern __shared__ int dyn[];
    __shared__ Shared sh;
    int *s_takes = dyn, *s_pieces = dyn + p.n + 1, *s_len = s_pieces + p.n + 1;         // [n + 1] each
    uint32_t *s_child = (uint32_t *)(s_len + p.n + 1);                                   // a bit a sequence
    const cg::cluster_group cl = cg::this_cluster();
    auto here = cl.barrier_arrive();
    const Parts parts(p.N, gridDim.x * blockDim.x / 32);
    const int tid = threadIdx.x, block = blockDim.x;
    const int thread = blockIdx.x * block + tid, threads = gridDim.x * block;       // of the cluster
    const int w = (tid >> 5) * gridDim.x + blockIdx.x, warps = threads >> 5;
    pdl_wait();
    pdl_trigger();
    if (tid == 0) sh.flags = 0;
    for (int i = tid; i < (p.S + 31) / 32; i += block) s_child[i] = 0;
    __syncthreads();
    Three sum = {0, 0, 0};
    int flags = 0, a = tid < p.n ? p.parents[tid] : 0, c = tid < p.n ? p.children[tid] : 0;
    count_free(p, sh, parts, w);             // while these are on their way
    for (int i0 = 0; i0 < p.n; i0 += block) {
        const int i = i0 + tid;
        int len = 0;
        if (i < p.n) {
            if (a < 0 || a >= p.S || c < 0 || c >= p.S) {
                flags |= FLAG_BAD_LENGTH;
            } else {
                const int most = p.lens[a];
                len = p.fork_lens ? p.fork_lens[i] : most;
                const uint32_t bit = 1u << (c & 31);
                // an empty sequence, and each but once
                if (most < 0 || most > p.cap || len < 0 || len > most || p.lens[c] != 0 ||
                    (atomicOr(&s_child[c / 32], bit) & bit)) {
                    flags |= FLAG_BAD_LENGTH;
                    len = 0;
                }
            }
        }
        if (i + block < p.n) {
            a = p.parents[i + block];
            c = p.children[i + block];
        }
        Three all;
        const Three at = scan_three({len % p.bs != 0, ceil_div(len / p.bs, kPiece), 0}, sh, all);
        if (i < p.n) {
            s_takes[i] = sum.x + at.x;
            s_pieces[i] = sum.y + at.y;
            s_len[i] = len;
        }
        sum = {sum.x + all.x, sum.y + all.y, 0};
    }
    const int takes = sum.x;
    if (tid == 0) {
        s_takes[p.n] = takes;
        s_pieces[p.n] = sum.y;
    }
    const auto common = [&](int i) { return make_int2(0, s_len[i] / p.bs); };
    // (sequences have been found in range)
    const auto sequence = [&](int i) { return min((unsigned)i, (unsigned)p.S - 1u); };
    const auto parent = [&](int i) { return p.table + (size_t)sequence(p.parents[i]) * p.W; };
    const auto child = [&](int i) { return p.table + (size_t)sequence(p.children[i]) * p.W; };
    if (!__syncthreads_or(flags)) {
        walk(s_pieces, p.n, w, warps, common, parent, [&](int, int, const int (&v)[kLane], int n) {
#pragma unroll
            for (int k = 0; k < kLane; ++k)
                if (k < n && (v[k] < 0 || v[k] >= p.N)) flags |= FLAG_BAD_BLOCK;
        });
        for (int i = thread; i < p.n; i += threads)
            if (s_len[i] % p.bs) {
                const int t = parent(i)[s_len[i] / p.bs];
                if (t < 0 || t >= p.N) flags |= FLAG_BAD_BLOCK;
            }
    }
    if (flags) atomicOr(&sh.flags, flags);
    const Totals t = exchange(cl, here, sh, w, warps, takes, 0);
    if (t.flags) {                           // nothing is changed
        if (thread == 0) {
            raise_flag(p.status, t.flags);
            *p.num_copies = 0;
            if (p.left) *p.left = t.all;
        }
        return;
    }
    hand_out(p, sh, parts, w, t.before, takes, [&](int r, int block) {
        const int i = find_seq(s_takes, p.n, r), j = s_len[i] / p.bs;
        p.copies[r] = make_int4(parent(i)[j], block, 0, s_len[i] % p.bs);
        child(i)[j] = block;
        p.ref[block] = 1;
    });
    // counts of blocks in use: no free one is mistaken for such a one, or the other way round
    walk(s_pieces, p.n, w, warps, common, parent, [&](int i, int j, const int (&v)[kLane], int n) {
        int32_t *to = child(i) + j;
#pragma unroll
        for (int k = 0; k < kLane; ++k)
            if (k < n && v[k] >= 0 && v[k] < p.N) {
                to[32 * k] = v[k];
                atomicAdd(&p.ref[v[k]], 1);
            }
    });
    for (int i = thread; i < p.n; i += threads) p.lens[sequence(p.children[i])] = s_len[i];
    if (thread == 0) {
        *p.num_copies = takes;
        if (p.left) *p.left = t.all - takes;
    }
}

// ---- compact ----------------------------------------------------------------

// Entries v of a table at at, at + 32, ..: those of moved blocks (none below `first`) follow.
__device__ __forceinline__ void follow(const PoolParams &p, int first, int32_t *at, const int (&v)[kLane], int n) {
    int to[kLane];
#pragma unroll
    for (int k = 0; k < kLane; ++k) to[k] = k < n && v[k] >= first && v[k] < p.N ? ~p.ref[v[k]] : -1;
#pragma unroll
    for (int k = 0; k < kLane; ++k)
        if (to[k] >= 0) at[32 * k] = to[k];
}

__global__ void __launch_bounds__(kMaxThreads, 1) compact_kernel(const PoolParams p) {
    extern __shared__ int dyn[];
    __shared__ Shared sh;
    int *s_pieces = dyn;                     // [S + 1]
    const cg::cluster_group cl = cg::this_cluster();
    auto here = cl.barrier_arrive();
    const Parts parts(p.N, gridDim.x * blockDim.x / 32);
    const int tid = threadIdx.x, block = blockDim.x, lane = tid & 31;
    const int thread = blockIdx.x * block + tid, threads = gridDim.x * block;       // of the cluster
    const int w = (tid >> 5) * gridDim.x + blockIdx.x, warps = threads >> 5;
    pdl_wait();
    pdl_trigger();
    if (tid == 0) sh.flags = 0;
    int pieces = 0, flags = 0, next = tid < p.S ? p.lens[tid] : 0;
    count_free(p, sh, parts, w);             // while these are on their way
    for (int b0 = 0; b0 < p.S; b0 += block) {
        const int b = b0 + tid;
        int len = next;
        next = b + block < p.S ? p.lens[b + block] : 0;
        if (len < 0 || len > p.cap) {
            flags |= FLAG_BAD_LENGTH;
            len = 0;
        }
        Three all;
        const Three at = scan_three({ceil_div(ceil_div(len, p.bs), kPiece), 0, 0}, sh, all);
        if (b < p.S) s_pieces[b] = pieces + at.x;
        pieces += all.x;
    }
    if (tid == 0) s_pieces[p.S] = pieces;
    const auto held = [&](int b) { return make_int2(0, ceil_div(p.lens[b], p.bs)); };
    const auto row = [&](int b) { return p.table + (size_t)b * p.W; };
    if (!__syncthreads_or(flags))            // lengths are fine: so are the ranges
        walk(s_pieces, p.S, w, warps, held, row, [&](int, int, const int (&v)[kLane], int n) {
#pragma unroll
            for (int k = 0; k < kLane; ++k)
                if (k < n && (v[k] < 0 || v[k] >= p.N)) flags |= FLAG_BAD_BLOCK;
        });
    if (flags) atomicOr(&sh.flags, flags);
    const Totals t = exchange(cl, here, sh, w, warps, 0, 0);
    const int live = p.N - t.all;
    if (t.flags) {
        if (thread == 0) {
            raise_flag(p.status, t.flags);
            *p.num_copies = 0;
            if (p.left) *p.left = live;
        }
        return;
    }
    // free blocks below `live`: those of the warps before the one with id `live`, and some of
    // that one's own. There are as many used blocks from `live` on.
    const int wl = min((int)((unsigned)live / (unsigned)parts.each), warps - 1);
    int holes = 0;
    for (int i = lane; i < wl; i += 32) holes += sh.free[i];
#pragma unroll 4
    for (int i0 = parts.begin(wl); i0 < live; i0 += 128) {
        const Free4 f = free4(p.ref, i0, live);
        holes += f.v[0] + f.v[1] + f.v[2] + f.v[3];
    }
    holes = __reduce_add_sync(0xffffffffu, holes);
    const int moves = min(holes, p.n);
    // the k-th used block from `live` on goes to the k-th free one below
    {
        const int lo = parts.begin(w), hi = parts.begin(w + 1);
        int rank = t.before;                 // free blocks before
        Free4 f = free4(p.ref, lo, hi);
        for (int i0 = lo; i0 < hi; i0 += 128) {
            const Free4 next = free4(p.ref, i0 + 128, hi);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t mask = __ballot_sync(0xffffffffu, f.v[k]);
                const int r = rank + __popc(mask & lanes_below()), i = i0 + 32 * k + lane;
                rank += __popc(mask);
                if (i >= hi) continue;
                if (i < live) {
                    if (f.v[k] && r < moves) p.copies[r].y = i;
                } else if (!f.v[k]) {
                    const int m = i - live - (r - holes);            // used blocks from `live` on before this one
                    if (m < moves) p.copies[m].x = i;
                }
            }
            f = next;
        }
    }
    cl.sync();
    // a moved block's count goes with it; where it was, where it went is noted for the tables
    for (int64_t i0 = thread; i0 < moves; i0 += 4 * threads) {
        int2 c[4];
        int count[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i0 + k * threads < moves) c[k] = *(const int2 *)(p.copies + i0 + k * threads);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i0 + k * threads < moves) count[k] = p.ref[c[k].x];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i0 + k * threads < moves) {
                *((int2 *)(p.copies + i0 + k * threads) + 1) = make_int2(0, p.bs);
                p.ref[c[k].y] = count[k];
                p.ref[c[k].x] = ~c[k].y;
            }
    }
    if (thread == 0) {
        *p.num_copies = moves;
        if (p.left) *p.left = live;
    }
    cl.sync();
    walk(s_pieces, p.S, w, warps, held, row, [&](int b, int j, const int (&v)[kLane], int n) {
        follow(p, live, p.table + (size_t)b * p.W + j, v, n);
    });
    cl.sync();
    for (int i = thread; i < moves; i += threads) p.ref[p.copies[i].x] = 0;
}

// The cluster, for `rows` rows of the table. A CTA alone is launched without one, and its barriers
// cost little: a step of 16 sequences, 1000 entries and 700 blocks takes 4.2 us with 512 threads,
// 4.8 with 1024, 5.6 with two CTAs of 512; compaction of them 5.0, 5.7, 8.0. Turnover of 64 sequences,
// 4300 entries and 2600 blocks: 9.9, 8.2, 8.7; compaction 10.4, 9.0, 10.4 (8 CTAs 8.9). With 16k entries and
// 12k blocks compaction takes 9.3 us with 8 CTAs of 512, 10.4 with 8 of 1024, 13.1 with one; with 33k and
// 24k 17.4, 14.0 and 50 (16 CTAs 12.5). Turnover of 512 sequences, 580k entries and 320k blocks: 33.5 us
// with 8 of 1024, 21.2 with 16, 196 with one.
struct Cluster {
    unsigned ctas, threads;
};
Cluster cluster_of(const PoolParams &p, int32_t rows) {
    const int64_t n = (int64_t)rows * p.W + p.N;
    if (n <= 12288) return {1, n <= 4096 ? 512u : 1024u};
    return {n <= 131072 ? 8u : 16u, n <= 32768 ? 512u : 1024u};
}

// Bytes of shared memory for n sequences (forks: n forks among S sequences).
constexpr size_t resize_smem(size_t S) { return 3 * sizeof(int) * (S + 1) + S; }
constexpr size_t fork_smem(size_t n, size_t S) { return 3 * sizeof(int) * (n + 1) + sizeof(uint32_t) * ((S + 31) / 32); }
constexpr size_t compact_smem(size_t S) { return sizeof(int) * (S + 1); }

static_assert(resize_smem(kPoolMax) + sizeof(Shared) <= 227 * 1024 && fork_smem(kPoolMax, kPoolMax) + sizeof(Shared) <= 227 * 1024,
              "a CTA's shared memory");

// most: the kernel's smem at its largest. The limit is the kernel's, for every thread of the process: all
// of them set it to this, since a smaller one, set between another thread's and its launch, would have that
// launch refused.
cudaError_t launch(void (*kern)(PoolParams), const PoolParams &p, Cluster c, size_t smem, size_t most, cudaStream_t st) {
    if (smem > 24576) {                      // with the static part, more than a launch may have without asking
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e != cudaSuccess) return e;
    }
    if (c.ctas > 8) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c.ctas);
    cfg.blockDim = dim3(c.threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = c.ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = c.ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_pool_resize(const PoolParams &p, cudaStream_t st) {
    return launch(resize_kernel, p, cluster_of(p, p.S), resize_smem(p.S), resize_smem(kPoolMax), st);
}
cudaError_t launch_pool_fork(const PoolParams &p, cudaStream_t st) {
    return launch(fork_kernel, p, cluster_of(p, p.n), fork_smem(p.n, p.S), fork_smem(kPoolMax, kPoolMax), st);
}
cudaError_t launch_pool_compact(const PoolParams &p, cudaStream_t st) {
    return launch(compact_kernel, p, cluster_of(p, p.S), compact_smem(p.S), compact_smem(kPoolMax), st);
}

}  // namespace mla
