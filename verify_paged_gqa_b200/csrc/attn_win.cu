// attn_win.cu -- sliding-window attention with sinks for blocks of up to 16
// query rows per KV head: decode, draft-verify windows, short prompt chunks.
//
// A window bounds what a block reads (window + sinks positions), so such a
// call is short, and what counts is that every SM has loads in flight soon and
// that nothing follows them.  One launch:
//
//   split    a unit (stream, KV head, row block) is one cluster of C thread
//            blocks, one block to an SM, each with a run of the unit's tiles.
//            C comes from the host's arguments (win_cluster_size).
//   loads    a producer warp fills a ring of 192 KB with TMA boxes: units of a
//            tile's positions x 128 dims (two boxes of 64 dims, 128-byte
//            swizzle), K of every slice of 128 dims, then V.  A tile is 128
//            positions (64 at head dim 512, so that 1.5 tiles fit).  Tiles are
//            assembled from page pieces (ring.cuh), and rows between the
//            sinks and the window, or past the stream's end, are not loaded.
//            (Fragments copied by the lanes with cp.async instead spent 55% of
//            a warp's time on issuing the copies: 12 streams x 4,100 positions
//            47 us.)
//   products eight consumer warps, each with 16 positions of a tile at a time:
//            mma.sync m16n8k16 with positions, then dims, on the 16 rows of A
//            and query rows on the 8 columns of B: S^T = K Q^T, O^T = V^T P^T, so
//            a decode block of up to 8 rows fills the instruction, and a warp
//            needs nothing from another until the end.  The order of a
//            contraction's terms is free, so dims are permuted to make each
//            lane's fragment 16 contiguous bytes of a K row, and output dims to
//            make it 16 contiguous bytes of a V row; positions are permuted so
//            that eight lanes' rows fall on all banks of the swizzled tile.  P
//            goes from one layout to the other with 8 x 8 transposes in
//            registers, in three bf16 parts (24 bits), and each product is
//            added to O in fp32 with rounding (the tensor cores truncate their
//            sums: chained over 2,048 positions that was 6e-6 of the output's
//            norm; now 3e-7).
//   join     each warp leaves its O, the groups of warps their maxima and sums
//            in shared memory; after one cluster barrier the cluster's blocks
//            combine them over distributed shared memory, each a share of the
//            output.
//
// D = 256 and 512: the warps are split over D / 128 slices of the dims as well;
// the warps that share positions sum their scores through shared memory.
#include "launch.cuh"
#include "ring.cuh"

#include <algorithm>

namespace tfp {

namespace {

constexpr int kConsumers = 8;                       // warps; one more produces
constexpr int kWinThreads = 32 * (kConsumers + 1);
constexpr int kChunk = 16;                          // positions a warp takes at a time
constexpr uint32_t kRingBytes = 196608;
constexpr float kRescaleLog2 = 8.f;                 // move a row's reference max only past this growth

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit values, two neighbours of a row per lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t a)
{
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The shared-memory address `addr` of the cluster's block `rank`.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, int rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ float peer_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ float4 peer_f32x4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

// Two probabilities as three bf16 pairs, each rounded to nearest: p = hi + mid
// + lo to 2^-26 p.
__device__ __forceinline__ void split3(float p0, float p1, uint32_t &hi, uint32_t &mid, uint32_t &lo)
{
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(p1), "f"(p0));
    const float r0 = p0 - bf_lo(hi), r1 = p1 - bf_hi(hi);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(mid) : "f"(r1), "f"(r0));
    const float q0 = r0 - bf_lo(mid), q1 = r1 - bf_hi(mid);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(q1), "f"(q0));
}

template <int D>
struct WinShape {
    static constexpr int T = D == 512 ? 64 : 128;             // positions of a tile
    static constexpr int kSlices = D / 128;
    static constexpr int kGroups = kConsumers / kSlices;      // groups of warps with the same positions
    static constexpr int CW = T / kChunk / kGroups;           // chunks of a tile per warp
    static constexpr uint32_t kBox = T * 128, kUnit = 2 * kBox;
    static constexpr int NU = kRingBytes / kUnit;             // ring units
    static constexpr int kHeights = D == 512 ? 7 : 8;         // boxes of 1, 2, 4, ..., T rows
    static_assert(NU >= 2 * kSlices, "a tile's K and V units fit the ring");
};

template <int D, int NT>
struct WinSmem {
    using W = WinShape<D>;
    // at the end, the consumer warps' unnormalised outputs [8 NT rows][128]
    alignas(1024) uint8_t ring[W::NU][W::kUnit];
    // the slices' partial scores, by parity of the tile
    alignas(16) float s[W::kSlices > 1 ? 2 : 1][W::kSlices > 1 ? kConsumers : 1][W::CW][32][4 * NT];
    float m[W::kGroups][8 * NT];   // reference maxima, log2 units
    float l[W::kGroups][8 * NT];   // sums
    uint64_t full[W::NU];
    uint64_t empty[W::NU];
    volatile int abort_flag;
    long long wait_limit;
};

template <int D, int NT>
constexpr size_t win_smem_bytes()
{
    return sizeof(WinSmem<D, NT>) + 1024;  // + alignment slack
}

template <int D>
struct WinArgs {
    WinParams p;
    CUtensorMap kmap[WinShape<D>::kHeights];
    CUtensorMap vmap[WinShape<D>::kHeights];
};

// The unit's piece of this block: tiles [t0, t1) of squeezed positions.
struct Piece {
    WorkItem it;
    int t0, t1;
};

// One page's rows of a tile: rows [row, row + n) come from pool rows y on.
struct Rows {
    int row, n, y;
};

// Piece i of a tile (its pages in order, those of the run before the skipped
// positions first); n = 0 past the last one.
__device__ __forceinline__ Rows tile_piece(const WinParams &p, const Piece &pc, const int32_t *trow, int tpos,
                                           int nvalid, int i, int *pieces)
{
    const TileRows rows = tile_rows(p, pc.it, tpos, nvalid);
    const int pos_b = tpos + rows.b + pc.it.skip;
    const int lp_a = tpos / p.P, lp_b = pos_b / p.P;
    const int off_a = tpos - lp_a * p.P, off_b = pos_b - lp_b * p.P;
    const int n_a = rows.a > 0 ? (off_a + rows.a - 1) / p.P + 1 : 0;
    const int n_b = nvalid > rows.b ? (off_b + nvalid - rows.b - 1) / p.P + 1 : 0;
    *pieces = n_a + n_b;
    Rows x = {0, 0, 0};
    if (i < n_a + n_b) {
        const bool first = i < n_a;
        const int k = first ? i : i - n_a;
        const int off = first ? off_a : off_b;
        const int slot = k == 0 ? off : 0;
        x.row = (first ? 0 : rows.b) + (k == 0 ? 0 : k * p.P - off);
        x.n = min((first ? rows.a : nvalid) - x.row, p.P - slot);
        int page = __ldg(trow + (first ? lp_a : lp_b) + k);
        if (page < 0 || page >= p.n_pages) {
            // never read: page 0 stands in (the stream's outputs are flagged)
            set_flag(p.flags, kDevBadPage);
            page = 0;
        }
        x.y = (page * p.Hkv + pc.it.kh) * p.P + slot;
    }
    return x;
}

// The whole producer warp: lane i copies piece i of every tile (a tile in
// pages of fewer than 4 positions has more than 32: the lanes go round).
template <int D, int NT>
__device__ __forceinline__ void win_producer(const WinArgs<D> &a, WinSmem<D, NT> &sm, const Piece &pc, int lane)
{
    using W = WinShape<D>;
    const WinParams &p = a.p;
    // row blocks of a unit read the same pages: keep them in L2 for each other
    uint64_t pol;
    if (p.n_rblk > 1)
        asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
    else
        pol = l2_evict_first_policy();
    const int32_t *trow = p.table + (int64_t)pc.it.s * p.table_stride;
    auto nvalid = [&](int t) { return min(W::T, pc.it.len - t * W::T); };
    uint32_t U = 0;  // units issued
    bool ok = true;
    int pieces, pieces_next = 0;
    Rows now = tile_piece(p, pc, trow, pc.t0 * W::T, nvalid(pc.t0), lane, &pieces);
    for (int t = pc.t0; ok && t < pc.t1; ++t) {
        // (the next tile's page ids are read while this one's units wait for room)
        Rows next = now;
        if (t + 1 < pc.t1)
            next = tile_piece(p, pc, trow, (t + 1) * W::T, nvalid(t + 1), lane, &pieces_next);
        const TileRows rows = tile_rows(p, pc.it, t * W::T, nvalid(t));
        const uint32_t bytes = (uint32_t)(rows.a + nvalid(t) - rows.b) * 256u;
#pragma unroll 1
        for (int x = 0; x < 2 * W::kSlices; ++x) {
            const int st = (int)(U % W::NU);
            if (lane == 0) {
                ok = pwait(sm, &sm.empty[st], ((U / W::NU) & 1u) ^ 1u, p.flags, kWaitEmpty);
                if (ok)
                    mbar_arrive_expect_tx(&sm.full[st], bytes);
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok)
                break;
            const CUtensorMap *maps = x < W::kSlices ? a.kmap : a.vmap;
            const int dim = 128 * (x % W::kSlices);
            Rows cur = now;
            for (int i = lane;;) {
                // one box for each set bit of n
                while (cur.n > 0) {
                    const int h = 31 - __clz(cur.n);
                    uint8_t *dst = sm.ring[st] + cur.row * 128;
                    tma_load_2d(dst, &maps[h], dim, cur.y, &sm.full[st], pol);
                    tma_load_2d(dst + W::kBox, &maps[h], dim + 64, cur.y, &sm.full[st], pol);
                    cur.row += 1 << h;
                    cur.y += 1 << h;
                    cur.n -= 1 << h;
                }
                i += 32;
                if (i >= pieces)
                    break;
                int again;
                cur = tile_piece(p, pc, trow, t * W::T, nvalid(t), i, &again);
            }
            __syncwarp();
            ++U;
        }
        now = next;
        pieces = pieces_next;
    }
    if (lane == 0) {
        // let the copies in flight land before the block can exit
        for (uint32_t k = 1; k <= (U < (uint32_t)W::NU ? U : (uint32_t)W::NU); ++k)
            (void)mbar_wait(&sm.full[(U - k) % W::NU], ((U - k) / W::NU) & 1u, sm.wait_limit);
    }
    __syncwarp();
}

// NT: tiles of 8 query rows.
template <int D, int NT>
__global__ void __launch_bounds__(kWinThreads, 1) attn_win_kernel(const __grid_constant__ WinArgs<D> a)
{
    using W = WinShape<D>;
    constexpr int R = 8 * NT;  // rows of a block (p.RB)
    constexpr int CW = W::CW;
    extern __shared__ uint8_t smem_raw[];
    WinSmem<D, NT> &sm = *reinterpret_cast<WinSmem<D, NT> *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const WinParams &p = a.p;
    const float NEG_INF = -__int_as_float(0x7f800000);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int C = p.whole, rank = blockIdx.x % C;
    int u = blockIdx.x / C;
    Piece pc;
    pc.it.b = u % p.n_rblk;
    u /= p.n_rblk;
    pc.it.kh = u % p.Hkv;
    pc.it.s = u / p.Hkv;
    const int s = pc.it.s, kh = pc.it.kh, m0 = pc.it.b * R, n_rows = min(p.M - m0, R);
    allow_dependent_launch();
    if (threadIdx.x == 0) {
        for (int k = 0; k < W::NU; ++k) {
            mbar_init(&sm.full[k], 1);
            mbar_init(&sm.empty[k], W::kGroups);
        }
        sm.abort_flag = 0;
        sm.wait_limit = p.wait_limit;
        fence_mbar_init();
    }
    if (warp == kConsumers && lane < W::kHeights) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&a.kmap[lane])) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&a.vmap[lane])) : "memory");
    }
    wait_prior_grid();
    __syncthreads();

    const int len = __ldg(p.lens + s);
    // output (and query) row of the block's row r
    auto row_of = [&](int r) {
        const int m = m0 + r, w = m / p.G;
        return ((int64_t)s * p.W + w) * p.Hq + kh * p.G + (m - w * p.G);
    };
    if (!len_ok(p, len)) {
        if (rank == 0) {
            if (threadIdx.x == 0)
                set_flag(p.flags, kDevBadLen);
            const float nan = __int_as_float(0x7fc00000);
            for (int e = threadIdx.x; e < n_rows * (D / 4); e += kWinThreads)
                *reinterpret_cast<float4 *>(p.out + row_of(e / (D / 4)) * D + e % (D / 4) * 4) =
                    make_float4(nan, nan, nan, nan);
        }
        return;  // (the whole cluster)
    }
    pc.it.len = len;
    set_window(p, pc.it);  // len and everything below in squeezed positions
    const int lim = block_lim(p, len, pc.it.b);
    const int n_tiles = (lim + W::T - 1) / W::T;
    pc.t0 = piece_start(n_tiles, rank, C);
    pc.t1 = piece_start(n_tiles, rank + 1, C);

    const int slice = warp % W::kSlices, group = warp / W::kSlices;
    const int g = lane >> 2, t = lane & 3;  // mma fragment coordinates
    // o[4 c + k][y][2 d + e]: dim 64 c + 8 g + 2 k + d of row 8 y + 2 t + e
    float o[8][NT][4];
    float mref[NT][2], l[NT][2];
    if (warp == kConsumers) {
        if (pc.t0 < pc.t1)
            win_producer<D, NT>(a, sm, pc, lane);
    } else {
        // the block's query rows 8 y + g, in the layout of K's
        uint4 qf[NT][4];
#pragma unroll
        for (int y = 0; y < NT; ++y) {
            const bool there = g + 8 * y < n_rows;
            const uint4 *src =
                reinterpret_cast<const uint4 *>(p.q + (there ? row_of(g + 8 * y) : 0) * D + slice * 128 + 8 * t);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                qf[y][c] = there ? __ldg(src + 4 * c) : make_uint4(0, 0, 0, 0);
        }
        // one past the last position that row 8 y + 2 t + e sees
        int end[NT][2];
#pragma unroll
        for (int y = 0; y < NT; ++y)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                end[y][e] = row_lim(p, pc.it.len, m0 + 8 * y + 2 * t + e);
                mref[y][e] = NEG_INF;
                l[y][e] = 0.f;
            }
        // chunks that every row of the block sees whole need no mask
        const int all_end = row_lim(p, pc.it.len, m0), all_begin = lim - p.window;
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int y = 0; y < NT; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[k][y][e] = 0.f;

        // K: the lane's rows are positions pk and pk + 8 of a chunk (A's rows g and
        // g + 8), V: positions 2 t and pv of each half (A's columns 2 t and 2 t + 1):
        // A's odd rows are positions shifted by 4, so that eight lanes' 16 bytes
        // lie on different banks
        const int pk = g & 1 ? g ^ 4 : g, pv = (2 * t + 1) ^ 4;
        bool ok = true;
        uint32_t U = 0;  // first unit of the tile
        for (int tile = pc.t0; ok && tile < pc.t1; ++tile, U += 2 * W::kSlices) {
            const int p0 = tile * W::T + group * CW * kChunk;  // the warp's first position
            // ---- S^T = K Q^T: x[i][y][2 h + e] is position p0 + 16 i + 8 h + pk, row 8 y + 2 t + e
            float x[CW][NT][4];
            {
                const uint32_t uk = U + slice;
                const int st = (int)(uk % W::NU);
                ok = pwait(sm, &sm.full[st], (uk / W::NU) & 1u, p.flags, kWaitFull);
                const uint8_t *kt = sm.ring[st] + (group * CW * kChunk + pk) * 128;
#pragma unroll
                for (int i = 0; i < CW; ++i) {
                    uint4 k[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            k[h][c] = *reinterpret_cast<const uint4 *>(kt + (c >> 1) * W::kBox + (16 * i + 8 * h) * 128 +
                                                                       (((4 * (c & 1) + t) ^ pk) << 4));
                    // two chains of sums per tile of rows
                    float z[NT][2][4];
#pragma unroll
                    for (int y = 0; y < NT; ++y)
#pragma unroll
                        for (int f = 0; f < 2; ++f)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                z[y][f][e] = 0.f;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int y = 0; y < NT; ++y) {
                            mma16816(z[y][0], k[0][c].x, k[1][c].x, k[0][c].y, k[1][c].y, qf[y][c].x, qf[y][c].y);
                            mma16816(z[y][1], k[0][c].z, k[1][c].z, k[0][c].w, k[1][c].w, qf[y][c].z, qf[y][c].w);
                        }
#pragma unroll
                    for (int y = 0; y < NT; ++y)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[i][y][e] = z[y][0][e] + z[y][1][e];
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm.empty[st]);
            }
            if constexpr (W::kSlices > 1) {
                // sum over the slices, in one order for all of the group's warps
                auto &xs = sm.s[tile & 1];
#pragma unroll
                for (int i = 0; i < CW; ++i)
#pragma unroll
                    for (int y = 0; y < NT; ++y)
                        *reinterpret_cast<float4 *>(&xs[warp][i][lane][4 * y]) =
                            make_float4(x[i][y][0], x[i][y][1], x[i][y][2], x[i][y][3]);
                named_barrier(1 + group, 32 * W::kSlices);
#pragma unroll
                for (int i = 0; i < CW; ++i)
#pragma unroll
                    for (int y = 0; y < NT; ++y) {
                        float4 b = *reinterpret_cast<const float4 *>(&xs[group * W::kSlices][i][lane][4 * y]);
#pragma unroll
                        for (int w = 1; w < W::kSlices; ++w) {
                            const float4 v =
                                *reinterpret_cast<const float4 *>(&xs[group * W::kSlices + w][i][lane][4 * y]);
                            b.x += v.x;
                            b.y += v.y;
                            b.z += v.z;
                            b.w += v.w;
                        }
                        x[i][y][0] = b.x;
                        x[i][y][1] = b.y;
                        x[i][y][2] = b.z;
                        x[i][y][3] = b.w;
                    }
            }
            // ---- masked scores in log2 units; does some row's maximum grow too far?
            const bool whole = p0 + CW * kChunk <= all_end && (p0 >= all_begin || p0 + CW * kChunk <= p.sinks);
            bool grow = false;
#pragma unroll
            for (int i = 0; i < CW; ++i)
#pragma unroll
                for (int y = 0; y < NT; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = x[i][y][e] * p.scale_log2;
                        if (!whole) {
                            // (positions that were not loaded are seen by no row)
                            const int pos = p0 + 16 * i + 8 * (e >> 1) + pk, n = end[y][e & 1];
                            if (pos >= n || (pos < n - p.window && pos >= p.sinks))
                                v = NEG_INF;
                        }
                        x[i][y][e] = v;
                        grow = grow || v > mref[y][e & 1] + kRescaleLog2;
                    }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int y = 0; y < NT; ++y) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = NEG_INF;
#pragma unroll
                        for (int i = 0; i < CW; ++i)
                            mx = fmax3(mx, x[i][y][e], x[i][y][2 + e]);
#pragma unroll
                        for (int k = 4; k < 32; k <<= 1)
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
                        const float m_new = fmaxf(mref[y][e], mx);
                        const float alpha = mref[y][e] == NEG_INF ? 0.f : fast_exp2(mref[y][e] - m_new);
                        mref[y][e] = m_new;
                        l[y][e] *= alpha;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            o[k][y][e] *= alpha;
                            o[k][y][2 + e] *= alpha;
                        }
                    }
                }
            }
            const uint32_t uv = U + W::kSlices + slice;
            const int st = (int)(uv % W::NU);
            const uint8_t *vt = sm.ring[st] + group * CW * kChunk * 128;
#pragma unroll
            for (int i = 0; i < CW; ++i) {
                // ---- P^T in three parts: part[y][f][h] holds A's columns 2 t, 2 t + 1 of half h, row 8 y + g
                uint32_t part[NT][3][2];
#pragma unroll
                for (int y = 0; y < NT; ++y) {
                    const float n0 = mref[y][0] == NEG_INF ? 0.f : -mref[y][0];
                    const float n1 = mref[y][1] == NEG_INF ? 0.f : -mref[y][1];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float a0 = fast_exp2(x[i][y][2 * h] + n0), a1 = fast_exp2(x[i][y][2 * h + 1] + n1);
                        l[y][0] += a0;
                        l[y][1] += a1;
                        split3(a0, a1, part[y][0][h], part[y][1][h], part[y][2][h]);
#pragma unroll
                        for (int f = 0; f < 3; ++f)
                            part[y][f][h] = transpose8(part[y][f][h]);
                    }
                }
                // ---- O^T += V^T P^T
                if (i == 0)
                    ok = pwait(sm, &sm.full[st], (uv / W::NU) & 1u, p.flags, kWaitFull) && ok;
                // rows that were not loaded hold anything (0 * NaN = NaN)
                bool there[4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int pos = p0 + 16 * i + 8 * (h >> 1) + (h & 1 ? pv : 2 * t);
                    there[h] = whole || (pos < pc.it.len && (pos < pc.it.sink_end || pos >= pc.it.dead_end));
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint4 v[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const int r = h & 1 ? pv : 2 * t;
                        v[h] = *reinterpret_cast<const uint4 *>(vt + c * W::kBox + (16 * i + 8 * (h >> 1) + r) * 128 +
                                                                ((g ^ r) << 4));
                        if (!whole && !there[h])
                            v[h] = make_uint4(0, 0, 0, 0);
                    }
                    float acc[4][NT][4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int y = 0; y < NT; ++y)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                acc[k][y][e] = 0.f;
#pragma unroll
                    for (int f = 2; f >= 0; --f) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            // (dims 2 k and 2 k + 1 of the lane's eight, by pairs of positions)
                            const uint32_t v0 = (&v[0].x)[k], v1 = (&v[1].x)[k], v2 = (&v[2].x)[k], v3 = (&v[3].x)[k];
                            const uint32_t a0 = __byte_perm(v0, v1, 0x5410), a1 = __byte_perm(v0, v1, 0x7632);
                            const uint32_t a2 = __byte_perm(v2, v3, 0x5410), a3 = __byte_perm(v2, v3, 0x7632);
#pragma unroll
                            for (int y = 0; y < NT; ++y)
                                mma16816(acc[k][y], a0, a1, a2, a3, part[y][f][0], part[y][f][1]);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int y = 0; y < NT; ++y)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                o[4 * c + k][y][e] += acc[k][y][e];
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sm.empty[st]);
        }
    }

    // ---- join: O by warp, maxima and sums by group ------------------------------
    __syncthreads();  // every unit was consumed: the ring is free
    if (warp < kConsumers) {
        float(*const o_part)[128] = reinterpret_cast<float(*)[128]>(&sm.ring[0][0] + warp * R * 512);
#pragma unroll
        for (int y = 0; y < NT; ++y) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int k = 4; k < 32; k <<= 1)
                    l[y][e] += __shfl_xor_sync(0xffffffffu, l[y][e], k);
                const int r = 8 * y + 2 * t + e;
                if (slice == 0 && g == 0) {
                    sm.m[group][r] = mref[y][e];
                    sm.l[group][r] = l[y][e];
                }
                if (r < n_rows) {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int k = 0; k < 4; k += 2)
                            *reinterpret_cast<float4 *>(&o_part[r][64 * c + 8 * g + 2 * k]) =
                                make_float4(o[4 * c + k][y][e], o[4 * c + k][y][2 + e], o[4 * c + k + 1][y][e],
                                            o[4 * c + k + 1][y][2 + e]);
                }
            }
        }
    }
    cluster_sync();
    const uint32_t m_addr = smem_addr(sm.m), l_addr = smem_addr(sm.l), o_addr = smem_addr(sm.ring);
    for (int e = rank * kWinThreads + threadIdx.x; e < n_rows * (D / 4); e += C * kWinThreads) {
        const int r = e / (D / 4), d = e % (D / 4) * 4;
        float top = NEG_INF;
        for (int k = 0; k < C; ++k)
#pragma unroll
            for (int w = 0; w < W::kGroups; ++w)
                top = fmaxf(top, peer_f32(peer_addr(m_addr, k) + (w * R + r) * 4));
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
        for (int k = 0; k < C; ++k) {
#pragma unroll
            for (int w = 0; w < W::kGroups; ++w) {
                const uint32_t at = (w * R + r) * 4;
                // (a group without positions: 2^-inf = 0)
                const float wt = fast_exp2(peer_f32(peer_addr(m_addr, k) + at) - top);
                sum = fmaf(wt, peer_f32(peer_addr(l_addr, k) + at), sum);
                const float4 v = peer_f32x4(peer_addr(o_addr, k) + (w * W::kSlices + d / 128) * R * 512 +
                                            (r * 128 + d % 128) * 4);
                acc.x = fmaf(wt, v.x, acc.x);
                acc.y = fmaf(wt, v.y, acc.y);
                acc.z = fmaf(wt, v.z, acc.z);
                acc.w = fmaf(wt, v.w, acc.w);
            }
        }
        const float inv = 1.f / sum;
        *reinterpret_cast<float4 *>(p.out + row_of(r) * D + d) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    }
    cluster_sync();  // no block leaves while others read its shared memory
}

// What a launch in clusters of C blocks looks like.
struct WinLaunch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];

    WinLaunch(int C, int grid, size_t bytes, cudaStream_t stream)
    {
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(kWinThreads);
        cfg.dynamicSmemBytes = bytes;
        cfg.stream = stream;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = C;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
    }
};

// Clusters of C blocks the current device holds at once (asked once per device).
template <int D, int NT>
int win_clusters(int C)
{
    static std::atomic<int> known[kMaxDevices][kMaxCluster + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return 0;
    int n = known[dev][C].load(std::memory_order_relaxed);
    if (n == 0) {
        constexpr size_t bytes = win_smem_bytes<D, NT>();
        static std::atomic<bool> configured[kMaxDevices];
        if (set_smem_limit_once(attn_win_kernel<D, NT>, bytes, configured) != cudaSuccess)
            return 0;
        WinLaunch launch(C, C, bytes, nullptr);
        launch.cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, attn_win_kernel<D, NT>, &launch.cfg) != cudaSuccess)
            return 0;
        known[dev][C].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <int D, int NT>
cudaError_t launch_win(const WinParams &p, int grid, cudaStream_t stream)
{
    constexpr size_t bytes = win_smem_bytes<D, NT>();
    static_assert(bytes <= 232448, "shared memory");
    static std::atomic<bool> configured[kMaxDevices];
    const cudaError_t e = set_smem_limit_once(attn_win_kernel<D, NT>, bytes, configured);
    if (e != cudaSuccess)
        return e;
    WinArgs<D> a;
    a.p = p;
    for (int h = 0; h < WinShape<D>::kHeights; ++h)
        if (!make_pool_map(&a.kmap[h], p.k_pool, p, 1 << h) || !make_pool_map(&a.vmap[h], p.v_pool, p, 1 << h))
            return cudaErrorInvalidValue;
    WinLaunch launch(p.whole, grid, bytes, stream);
    return cudaLaunchKernelEx(&launch.cfg, attn_win_kernel<D, NT>, a);
}

template <int NT>
cudaError_t launch_win_rows(const WinParams &p, int grid, cudaStream_t stream)
{
    return p.D == 128   ? launch_win<128, NT>(p, grid, stream)
           : p.D == 256 ? launch_win<256, NT>(p, grid, stream)
                        : launch_win<512, NT>(p, grid, stream);
}

template <int NT>
int win_clusters_rows(int D, int C)
{
    return D == 128 ? win_clusters<128, NT>(C) : D == 256 ? win_clusters<256, NT>(C) : win_clusters<512, NT>(C);
}

}  // namespace

// Blocks per cluster.  The blocks of one wave run side by side; a block's
// time is its tiles one after another, plus starting and joining (about
// kEntry tiles).  So: the cluster size whose waves times that is least (ties to
// the smaller).
int win_cluster_size(const WinParams &p, int64_t units)
{
    constexpr int kEntry = 4;
    const int64_t seen = std::min<int64_t>(p.max_len, (int64_t)p.window + p.sinks + p.W);
    const int T = p.D == 512 ? 64 : 128;
    const int64_t tiles = (seen + T - 1) / T;
    int best = 1;
    int64_t least = INT64_MAX;
    for (int C = 1; C <= kMaxCluster; ++C) {
        const int64_t at_once = p.RB == 8 ? win_clusters_rows<1>(p.D, C) : win_clusters_rows<2>(p.D, C);
        if (at_once <= 0)
            continue;
        const int64_t waves = (units + at_once - 1) / at_once;
        const int64_t cost = waves * ((tiles + C - 1) / C + kEntry);
        if (cost < least) {
            least = cost;
            best = C;
        }
    }
    return best;
}

cudaError_t launch_attn_win(const WinParams &p, int grid, cudaStream_t stream)
{
    return p.RB == 8 ? launch_win_rows<1>(p, grid, stream) : launch_win_rows<2>(p, grid, stream);
}

}  // namespace tfp
