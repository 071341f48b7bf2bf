// kv_pages.cu -- the cache's pages, shared by reference count: fork, grow,
// free and compact, and the page moves they ask for.
//
// TensorFold #1620, opening comment: a stream takes pages of the core pool as
// it grows and gives them back; kept states walk a slot's pages.  Here the
// pool's bookkeeping is one device array, refs[page]: how many table entries
// hold the page, 0 for a free one.  There is no free list: a page is taken by
// looking for the lowest free ids, so the outcome depends on refs and the
// tables alone, never on the order in which pages came back, and counts
// change by integer atomics, whose order does not show.
//
//   fork     child rows of a table name their parents' pages (refs + 1)
//   free     entries give their pages back (refs - 1) and hold -1
//   grow     every position that a step writes gets a page of its own: a fresh
//            one where the entry holds none, a copy where others share it
//   compact  the live pages move to ids 0 .. n_live - 1: the k-th live page at
//            or past n_live goes to the k-th free one below
//
// grow and compact only change the bookkeeping and leave a list of page moves
// {source, destination, positions}; pages_move performs it on one layer's pool
// (a model's layers share the table and have a pool each).  A list's
// destinations were free when it was made and its sources were held, so no page
// is both and the moves need no order.  A source of grow's may be free by then
// (every holder of a shared page took a copy): its contents last until the next
// call that changes refs, which is why the moves come first on every layer.
//
// The bookkeeping is a few kilobytes: a call's time is its latency, so each is
// one kernel (compact over a table of more than 4,096 entries has a second), 2 to
// 3 us.  grow and compact scan refs with one block of 1,024 threads, 4 counts a
// thread.  pages_move is bound by memory: 16 KB runs through a ring of four
// shared-memory stages with bulk copies (TMA engine) in both directions, three
// blocks to an SM (a compaction that moves 0.5 GB: 189 us with its bookkeeping,
// 5.8 TB/s read and written).  Where the free pages lie behind 95,000 held ones
// grow's scan takes 20 us, behind 950,000 188 us; compact reads all of refs twice
// (41 us for 100,000 pages, 354 for 1,000,000).
#include "launch.cuh"

namespace tfp {

namespace {

constexpr int kScanThreads = 1024;
constexpr int kScanPer = 4;                        // counts a thread takes at a time
constexpr int64_t kRetableHere = 4096;             // table entries that compact's own block rewrites
constexpr uint32_t kMoveChunk = 16384;             // bytes of one run
constexpr int kMoveStages = 4;
constexpr int kMoveBlocksPerSm = 3;

__device__ __forceinline__ void note(uint32_t *status, uint32_t bit)
{
    if (status)
        atomicOr(status, bit);
}

__device__ __forceinline__ int pages_of(int len, int P) { return (int)(((int64_t)len + P - 1) / P); }

// Drops one holder of page id; a page that nobody holds is reported and left.
__device__ __forceinline__ void release(const PagesParams &p, int id)
{
    if (atomicSub(p.refs + id, 1) <= 0) {
        atomicAdd(p.refs + id, 1);
        note(p.status, kDevBadPage);
    }
}

__global__ void __launch_bounds__(256) pages_fork_kernel(const __grid_constant__ PagesParams p)
{
    const int c = blockIdx.y;
    const int j = blockIdx.x * 256 + threadIdx.x;
    const int parent = __ldg(p.parents + c);
    int len = 0;
    if (parent >= 0 && parent < p.S) {
        len = __ldg(p.lens + parent);
        const int n = len < 0 ? 0 : pages_of(len, p.P);
        if (len < 0 || n > p.stride || n > p.dst_stride) {
            if (j == 0)
                note(p.status, kDevBadLen);
            len = 0;
        }
    } else if (parent != -1 && j == 0) {
        note(p.status, kDevBadLen);
    }
    if (j == 0)
        p.dst_lens[c] = len;
    if (j >= p.dst_stride)
        return;
    int id = -1;
    if (j < pages_of(len, p.P)) {
        id = p.table[(int64_t)parent * p.stride + j];
        if (id >= p.n_pages) {
            note(p.status, kDevBadPage);
            id = -1;
        }
        if (id >= 0) {
            // A page that nobody holds is not taken: its next owner would share
            // it.  (Counts only rise here, and only from 1 on, so a 0 is one
            // for every child that looks.)
            if (__ldcg(p.refs + id) <= 0) {
                note(p.status, kDevBadPage);
                id = -1;
            } else {
                atomicAdd(p.refs + id, 1);
            }
        }
    }
    p.dst_table[(int64_t)c * p.dst_stride + j] = id < 0 ? -1 : id;
}

// Entries [first, end) of every row give their pages back.
template <bool kWindow>
__global__ void __launch_bounds__(256) pages_free_kernel(const __grid_constant__ PagesParams p)
{
    const int s = blockIdx.y;
    const int j = blockIdx.x * 256 + threadIdx.x;
    int first = 0, end = p.stride;
    if constexpr (kWindow) {
        // a later row sits at position len or past it: it sees positions below
        // `sinks` and positions past len - window
        const int len = __ldg(p.lens + s);
        if (len < 0 || (int64_t)len > (int64_t)p.stride * p.P) {
            if (j == 0)
                note(p.status, kDevBadLen);
            return;
        }
        first = pages_of(p.sinks, p.P);
        end = len < p.window ? 0 : (len - p.window + 1) / p.P;
    } else {
        if (p.first)
            first = __ldg(p.first + s);
        if (p.end)
            end = __ldg(p.end + s);
        if (first < 0 || first > p.stride || end < 0 || end > p.stride) {
            if (j == 0)
                note(p.status, kDevBadLen);
            return;
        }
    }
    if (j < first || j >= end)
        return;
    int32_t *entry = p.table + (int64_t)s * p.stride + j;
    const int id = *entry;
    if (id < 0)
        return;
    if (id >= p.n_pages) {
        note(p.status, kDevBadPage);
        return;
    }
    *entry = -1;
    release(p, id);
}

// Exclusive prefix sum of v over the block's threads; *total gets the sum.
// The caller's next write to shared memory is ordered by the final barrier.
__device__ __forceinline__ int block_scan(int v, int *total)
{
    __shared__ int warp_sum[kScanThreads / 32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int incl = v;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const int got = __shfl_up_sync(0xffffffffu, incl, k);
        if (lane >= k)
            incl += got;
    }
    if (lane == 31)
        warp_sum[warp] = incl;
    __syncthreads();
    int w = warp_sum[lane];
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const int got = __shfl_up_sync(0xffffffffu, w, k);
        if (lane >= k)
            w += got;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) % 32);
    __syncthreads();
    return incl - v + (warp > 0 ? before : 0);
}

// refs[i .. i + 3] (past the end: a value that counts as neither free nor
// live), refs 16-byte aligned and i a multiple of 4.
__device__ __forceinline__ void load_refs(const PagesParams &p, int i, int (&r)[kScanPer])
{
    if (i + kScanPer <= p.n_pages) {
        const int4 v = *reinterpret_cast<const int4 *>(p.refs + i);
        r[0] = v.x;
        r[1] = v.y;
        r[2] = v.z;
        r[3] = v.w;
    } else {
#pragma unroll
        for (int e = 0; e < kScanPer; ++e)
            r[e] = i + e < p.n_pages ? p.refs[i + e] : -1;
    }
}

// One block.  Item (s, k): the k-th page that stream s's new rows touch.
__global__ void __launch_bounds__(kScanThreads, 1) pages_grow_kernel(const __grid_constant__ PagesParams p)
{
    const int64_t items = (int64_t)p.S * p.per_stream;
    // the items that need a page, in order: list entry k = {the page to copy
    // from or -1, -, positions to copy, item}
    int need = 0;
    for (int64_t i0 = 0; i0 < items; i0 += kScanThreads) {
        const int64_t i = i0 + threadIdx.x;
        int src = -1, n_pos = 0, entry = 0;
        bool wants = false;
        if (i < items) {
            const int s = (int)(i / p.per_stream), k = (int)(i - (int64_t)s * p.per_stream);
            const int len = __ldg(p.lens + s);
            if (len != 0 && (len < p.rows || (int64_t)len > (int64_t)p.stride * p.P)) {
                note(p.status, kDevBadLen);
            } else if (len != 0) {
                const int start = len - p.rows;  // the first new position
                const int j = start / p.P + k;
                if (j <= (len - 1) / p.P) {
                    entry = s * p.stride + j;  // (S * stride fits 31 bits)
                    const int id = p.table[entry];
                    if (id < 0) {
                        wants = true;
                    } else if (id >= p.n_pages || p.refs[id] <= 0) {
                        note(p.status, kDevBadPage);
                    } else if (p.refs[id] > 1) {
                        wants = true;
                        src = id;
                        n_pos = k == 0 ? start - j * p.P : 0;
                    }
                }
            }
        }
        int total;
        const int at = need + block_scan(wants ? 1 : 0, &total);
        if (wants)
            p.moves[1 + at] = make_int4(src, -1, n_pos, entry);
        need += total;
    }
    // the lowest free pages
    int found = 0;
    for (int i0 = 0; i0 < p.n_pages && found < need; i0 += kScanThreads * kScanPer) {
        const int i = i0 + threadIdx.x * kScanPer;
        int r[kScanPer], n = 0, total;
        load_refs(p, i, r);
#pragma unroll
        for (int e = 0; e < kScanPer; ++e)
            n += r[e] == 0;
        int at = found + block_scan(n, &total);
#pragma unroll
        for (int e = 0; e < kScanPer; ++e) {
            if (r[e] == 0) {
                if (at < need)
                    p.moves[1 + at].y = i + e;
                ++at;
            }
        }
        found += total;
    }
    __syncthreads();  // the list is complete (block scope: one block reads it)
    const bool enough = found >= need;
    if (threadIdx.x == 0) {
        p.moves[0] = make_int4(enough ? need : 0, 0, 0, 0);
        if (!enough)
            note(p.status, kDevNoPage);
    }
    if (!enough)
        return;  // nothing was changed
    for (int k = threadIdx.x; k < need; k += kScanThreads) {
        const int4 m = p.moves[1 + k];
        p.table[m.w] = m.y;
        p.refs[m.y] = 1;
        if (m.x >= 0)
            atomicSub(p.refs + m.x, 1);
    }
}

// Table entry i follows its page if that moved (the list's sources ascend:
// binary search among `moves` of them; pages below n_live stay).
__device__ __forceinline__ void retable(const PagesParams &p, int64_t i, int moves, int n_live)
{
    const int id = p.table[i];
    if (id < n_live)
        return;  // none, or a page that stays
    int lo = 0, hi = moves;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (p.moves[1 + mid].x < id)
            lo = mid + 1;
        else
            hi = mid;
    }
    if (lo < moves && p.moves[1 + lo].x == id)
        p.table[i] = p.moves[1 + lo].y;
    else
        note(p.status, kDevBadPage);  // nobody holds this page
}

// One block.
__global__ void __launch_bounds__(kScanThreads, 1) pages_compact_kernel(const __grid_constant__ PagesParams p)
{
    allow_dependent_launch();
    int live = 0;
    for (int i = threadIdx.x * kScanPer; i < p.n_pages; i += kScanThreads * kScanPer) {
        int r[kScanPer];
        load_refs(p, i, r);
#pragma unroll
        for (int e = 0; e < kScanPer; ++e)
            live += r[e] > 0;
    }
    int n_live;
    (void)block_scan(live, &n_live);
    // holes below n_live and live pages from n_live on: as many of the one as
    // of the other
    int holes = 0, movers = 0;
    for (int i0 = 0; i0 < p.n_pages; i0 += kScanThreads * kScanPer) {
        const int i = i0 + threadIdx.x * kScanPer;
        int r[kScanPer], h = 0, m = 0, total;
        load_refs(p, i, r);
#pragma unroll
        for (int e = 0; e < kScanPer; ++e) {
            h += i + e < n_live && r[e] <= 0;
            m += i + e >= n_live && r[e] > 0;
        }
        // (an iteration holds at most 4,096 of each: two sums in one scan)
        const int at = block_scan(h | (m << 16), &total);
        int ah = holes + (at & 0xffff), am = movers + (at >> 16);
#pragma unroll
        for (int e = 0; e < kScanPer; ++e) {
            if (i + e < n_live && r[e] <= 0)
                p.moves[1 + ah++].y = i + e;
            if (i + e >= n_live && r[e] > 0)
                p.moves[1 + am++].x = i + e;
        }
        holes += total & 0xffff;
        movers += total >> 16;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < movers; k += kScanThreads) {
        const int src = p.moves[1 + k].x, dst = p.moves[1 + k].y;
        p.moves[1 + k].z = p.P;
        p.moves[1 + k].w = 0;
        p.refs[dst] = p.refs[src];
        p.refs[src] = 0;
    }
    if (threadIdx.x == 0)
        p.moves[0] = make_int4(movers, n_live, 0, 0);
    const int64_t entries = (int64_t)p.S * p.stride;
    if (entries <= kRetableHere)
        for (int64_t i = threadIdx.x; i < entries; i += kScanThreads)
            retable(p, i, movers, n_live);
}

// Larger tables, by as many blocks as they need.
__global__ void __launch_bounds__(256) pages_retable_kernel(const __grid_constant__ PagesParams p)
{
    wait_prior_grid();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int4 head = p.moves[0];
    if (i < (int64_t)p.S * p.stride)
        retable(p, i, head.x, head.y);
}

// ---- the moves ---------------------------------------------------------------

struct Run {
    const uint8_t *src;
    uint8_t *dst;
    uint32_t bytes;  // 0: nothing to copy
};

// Chunk c of the list: the pieces of an entry vary slowest, so that the first
// pieces, which every entry has, spread over all blocks.
__device__ __forceinline__ Run run_of(const MoveParams &p, int64_t c, int count)
{
    Run run = {nullptr, nullptr, 0};
    const int e = (int)(c % count);
    int t = (int)(c / count);  // [0, 2 * pieces)
    const int4 m = *reinterpret_cast<const int4 *>(p.moves + 4 * (int64_t)(1 + e));
    const int n_pos = min(m.z, p.P);
    if (m.x < 0 || n_pos <= 0)
        return run;
    if (m.x >= p.n_pages || m.y < 0 || m.y >= p.n_pages) {
        if (t == 0)
            note(p.status, kDevBadPage);
        return run;
    }
    const bool is_v = t >= p.pieces;
    t -= is_v ? p.pieces : 0;
    const int64_t row = (int64_t)p.D * 2, head = p.P * row, page = p.Hkv * head;
    int64_t off, bytes;
    if (n_pos == p.P) {
        // the whole page is one run
        off = (int64_t)t * kMoveChunk;
        bytes = page - off;
    } else {
        // the first positions of each KV head
        const int kh = t / p.per_head;
        const int64_t o = (int64_t)(t - kh * p.per_head) * kMoveChunk;
        off = kh * head + o;
        bytes = n_pos * row - o;
    }
    if (bytes <= 0)
        return run;
    const uint8_t *base = reinterpret_cast<const uint8_t *>(is_v ? p.v_pool : p.k_pool);
    run.src = base + m.x * page + off;
    run.dst = const_cast<uint8_t *>(base) + m.y * page + off;
    run.bytes = bytes < kMoveChunk ? (uint32_t)bytes : kMoveChunk;
    return run;
}

// One lane per block walks its chunks: loads run three stages ahead of the
// stores.
__global__ void __launch_bounds__(32) pages_move_kernel(const __grid_constant__ MoveParams p)
{
    extern __shared__ __align__(128) uint8_t smem[];  // kMoveStages runs
    __shared__ uint64_t full[kMoveStages];
    wait_prior_grid();
    if (threadIdx.x != 0)
        return;
    const int count = min(p.moves[0], p.cap);
    if (count <= 0)
        return;
    for (int k = 0; k < kMoveStages; ++k)
        mbar_init(&full[k], 1);
    fence_mbar_init();
    const uint64_t pol = l2_evict_first_policy();
    const int64_t chunks = (int64_t)count * 2 * p.pieces;
    int64_t next = blockIdx.x;
    Run runs[kMoveStages];
    // the next run with bytes, loaded into stage `st`; false when none is left
    auto load = [&](int st) {
        for (; next < chunks; next += gridDim.x) {
            runs[st] = run_of(p, next, count);
            if (runs[st].bytes != 0) {
                next += gridDim.x;
                mbar_arrive_expect_tx(&full[st], runs[st].bytes);
                bulk_g2s(smem + st * kMoveChunk, runs[st].src, runs[st].bytes, &full[st], pol);
                return true;
            }
        }
        return false;
    };
    int issued = 0;
#pragma unroll
    for (int k = 0; k < kMoveStages - 1; ++k)
        issued += load(k) ? 1 : 0;
    bool ok = true;
    uint32_t parity = 0;
    int done = 0;
    while (ok && done < issued) {
#pragma unroll
        for (int st = 0; st < kMoveStages; ++st) {
            if (ok && done < issued) {
                ok = mbar_wait(&full[st], parity);
                if (ok) {
                    bulk_s2g(runs[st].dst, smem + st * kMoveChunk, runs[st].bytes);
                    bulk_commit();
                    ++done;
                    // the stage before this one is free once its store has read it
                    bulk_wait_read<1>();
                    issued += load((st + kMoveStages - 1) % kMoveStages) ? 1 : 0;
                }
            }
        }
        parity ^= 1u;
    }
    if (!ok) {
        note(p.status, kDevTimeout);
        for (int k = 0; k < kMoveStages; ++k)  // the copies in flight land before the block exits
            if (k < issued)
                (void)mbar_wait(&full[k], ((issued - 1 - k) / kMoveStages) & 1);
    }
    bulk_wait_all();
}

}  // namespace

cudaError_t launch_pages_fork(const PagesParams &p, int n_dst, cudaStream_t stream)
{
    for (int c0 = 0; c0 < n_dst; c0 += 65535) {
        PagesParams q = p;
        q.parents += c0;
        q.dst_table += (int64_t)c0 * p.dst_stride;
        q.dst_lens += c0;
        const int n = n_dst - c0 < 65535 ? n_dst - c0 : 65535;
        pages_fork_kernel<<<dim3((p.dst_stride + 255) / 256, n), 256, 0, stream>>>(q);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

cudaError_t launch_pages_free(const PagesParams &p, bool window, cudaStream_t stream)
{
    for (int s0 = 0; s0 < p.S; s0 += 65535) {
        PagesParams q = p;
        q.table += (int64_t)s0 * p.stride;
        q.lens = p.lens ? p.lens + s0 : nullptr;
        q.first = p.first ? p.first + s0 : nullptr;
        q.end = p.end ? p.end + s0 : nullptr;
        const dim3 grid((p.stride + 255) / 256, p.S - s0 < 65535 ? p.S - s0 : 65535);
        if (window)
            pages_free_kernel<true><<<grid, 256, 0, stream>>>(q);
        else
            pages_free_kernel<false><<<grid, 256, 0, stream>>>(q);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

cudaError_t launch_pages_grow(const PagesParams &p, cudaStream_t stream)
{
    pages_grow_kernel<<<1, kScanThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_pages_compact(const PagesParams &p, cudaStream_t stream)
{
    pages_compact_kernel<<<1, kScanThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    const int64_t entries = (int64_t)p.S * p.stride;
    if (e != cudaSuccess || entries <= kRetableHere)
        return e;
    return launch_dependent(pages_retable_kernel, dim3((unsigned)((entries + 255) / 256)), dim3(256), 0,
                            stream, p);
}

cudaError_t launch_pages_move(MoveParams p, int sms, cudaStream_t stream)
{
    const int64_t head = (int64_t)p.P * p.D * 2;
    p.per_head = (int)((head + kMoveChunk - 1) / kMoveChunk);
    const int64_t pieces = (int64_t)p.Hkv * p.per_head;
    const int64_t most = (int64_t)p.cap * 2 * pieces;
    if (pieces > 0x3fffffff)
        return cudaErrorInvalidValue;
    p.pieces = (int)pieces;
    if (most == 0)
        return cudaSuccess;
    static std::atomic<bool> configured[kMaxDevices];
    constexpr size_t bytes = kMoveStages * kMoveChunk;
    const cudaError_t e = set_smem_limit_once(pages_move_kernel, bytes, configured);
    if (e != cudaSuccess)
        return e;
    const int64_t grid = (int64_t)sms * kMoveBlocksPerSm;
    return launch_dependent(pages_move_kernel, dim3((unsigned)(most < grid ? most : grid)), dim3(32), bytes,
                            stream, p);
}

}  // namespace tfp
