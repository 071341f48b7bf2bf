// attn_win.cu -- sliding-window attention with sinks for blocks of up to 16
// query rows per KV head: decode, draft-verify windows, short prompt chunks.
//
// A window bounds what a block reads (window + sinks positions), so such a
// call is short and what counts is its latency and that every SM has loads in
// flight from the first microsecond on.  The kernel therefore has no producer
// warp, no ring that its warps share and no second launch:
//
//   split    a unit (stream, KV head, row block) is one cluster of C thread
//            blocks; its positions are dealt out in chunks of 16 to the
//            cluster's 4 C / (D / 128) teams of warps, chunk k to team k mod
//            (teams).  C comes from the host's arguments (launch rule below).
//   loads    asynchronous 16-byte copies into each warp's own ring in shared
//            memory, two or three chunks deep (192 KB in flight per SM): K by
//            fragments (a lane copies what it reads back, 512 contiguous bytes a
//            warp), V by rows.  Only rows that some query row sees are read;
//            pages cost one table lookup per position, a chunk ahead.
//   products S^T = K Q^T: mma.sync m16n8k16 with positions on the 16 rows of A and
//            query rows on the 8 columns of B, so a decode block of up to 8 rows
//            fills the instruction; the order of a contraction's terms is free,
//            so dims are permuted to make each lane's fragment 16 contiguous
//            bytes of a K row.
//            O += P V, up to 8 rows: packed fp32 FMAs over two rows, P in fp32
//            through shared memory; half a warp takes the even positions, the
//            other half the odd ones, eight dims a lane.  (mma.sync runs at a
//            quarter of its nominal rate here, 32 cycles per scheduler: with P
//            in three bf16 parts, for the same accuracy, PV took 192 cycles
//            per SM and chunk, these FMAs take 64.)
//            16 rows, whose sums would not fit the registers that way: O^T = V^T
//            P^T with mma.sync, P in three bf16 parts (24 bits) moved from one
//            fragment layout to the other by 8 x 8 transposes, V in fragments as
//            K; each chunk's product is added to O in fp32 with rounding (the
//            tensor cores truncate their sums: chained over 128 chunks that
//            was 6e-6 of the output's norm, now 3e-7).
//   join     each warp leaves its O, the teams their maxima and sums in shared
//            memory; after one cluster barrier the cluster's blocks combine
//            them over distributed shared memory, each a share of the output.
//
// Measured: 12 streams of 32 query heads over a window of 4,096 38.7 us (5.2 TB/s:
// one and a half waves of clusters, so the start and the join show), 64 ragged
// streams over windows up to 8,192 in pages of 64 180 us (5.4 TB/s of the
// positions they have), one stream and KV head over 256 positions 5.6 us.
//
// D = 256 and 512: a team is D / 128 warps that share positions and split the
// dims; the chunk's scores are summed over the team through shared memory.
#include "launch.cuh"
#include "plan.cuh"

#include <algorithm>

namespace tfp {

namespace {

constexpr int kWinThreads = 128;
constexpr int kWinWarps = kWinThreads / 32;
constexpr int kChunk = 16;               // positions a team takes at a time
// Blocks per SM and chunks in flight per warp: either way 192 KB in flight.
// (A warp's own chain of latencies bounds a chunk, so up to eight rows, whose
// registers allow it, run twelve warps on an SM.)
constexpr int win_blocks(int R) { return R <= 8 ? 3 : 2; }
constexpr int win_stages(int R) { return R <= 8 ? 2 : 3; }
constexpr float kRescaleLog2 = 8.f;      // move a row's reference max only past this growth

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Copies 16 bytes to shared memory asynchronously, or zeroes them (nothing is
// read then).
__device__ __forceinline__ void copy16(uint32_t dst, const __nv_bfloat16 *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}

// An 8 x 8 matrix of 16-bit values, two neighbours of a row per lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t a)
{
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Two probabilities as three bf16 pairs, each rounded to nearest: p = hi + mid
// + lo to 2^-26 p.
__device__ __forceinline__ void split3(float p0, float p1, uint32_t (&part)[3])
{
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(part[0]) : "f"(p1), "f"(p0));
    const float r0 = p0 - bf_lo(part[0]), r1 = p1 - bf_hi(part[0]);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(part[1]) : "f"(r1), "f"(r0));
    const float q0 = r0 - bf_lo(part[1]), q1 = r1 - bf_hi(part[1]);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(part[2]) : "f"(q1), "f"(q0));
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Waits until at most N of the thread's groups of copies are in flight.
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

template <int D, int R>
struct WinSmem {
    static constexpr int kTeam = D / 128;               // warps per team
    static constexpr int kTeams = kWinWarps / kTeam;
    // a warp's ring: [stage][K fragments [copy][lane], V rows [position][128]]; at
    // its end, the warp's unnormalised output [row][128]
    alignas(16) uint4 ring[kWinWarps][win_stages(R)][2][8][32];
    // the team's partial scores, by parity of the chunk
    alignas(16) float s[kTeam > 1 ? 2 : 1][kTeam > 1 ? kWinWarps : 1][kTeam > 1 ? 32 : 1][R == 16 ? 8 : 4];
    alignas(16) float p[kWinWarps][kChunk][R <= 8 ? R : 4];  // a warp's probabilities (FMAs)
    alignas(16) float alpha[kWinWarps][R <= 8 ? R : 4];      // factors of the last change of reference
    float m[kTeams][R];                                 // reference maxima, log2 units
    float l[kTeams][R];                                 // sums
};

// R: rows of a block (p.RB): 4, 8 or 16.
template <int D, int R>
__global__ void __launch_bounds__(kWinThreads, win_blocks(R)) attn_win_kernel(const __grid_constant__ WinParams p)
{
    constexpr int NT = R == 16 ? 2 : 1;  // tiles of 8 rows of the score product
    constexpr bool kMmaPv = R == 16;
    constexpr int kStages = win_stages(R);
    using Smem = WinSmem<D, R>;
    constexpr int kTeam = Smem::kTeam, kTeams = Smem::kTeams;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const float NEG_INF = -__int_as_float(0x7f800000);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int team = warp / kTeam, slice = warp % kTeam;  // slice: this warp's 128 dims
    const int g = lane >> 2, t = lane & 3;                // mma fragment coordinates
    const int C = p.whole, rank = blockIdx.x % C;
    int u = blockIdx.x / C;
    const int b = u % p.n_rblk;
    u /= p.n_rblk;
    const int kh = u % p.Hkv, s = u / p.Hkv;
    const int m0 = b * R, n_rows = min(p.M - m0, R);
    allow_dependent_launch();
    wait_prior_grid();

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
    // the positions that some row sees: [0, sink_end) and [start, lim), as
    // indexes [0, n)
    const int first = block_start(p, len, b);
    const int sink_end = first > p.sinks ? p.sinks : 0;
    const int start = first > p.sinks ? first : 0;
    const int lim = row_lim(p, len, m0 + R - 1);
    const int n = sink_end + lim - start;
    const int n_chunks = (n + kChunk - 1) / kChunk;
    const int shift = start - sink_end;  // position of index i >= sink_end: i + shift
    const int32_t *trow = p.table + (int64_t)s * p.table_stride;

    // the pool row of index 16 ch + (lane % 16), or -1
    auto lookup = [&](int ch) {
        const int i = ch * kChunk + (lane & 15);
        if (ch >= n_chunks || i >= n)
            return -1;
        const int pos = i < sink_end ? i : i + shift;
        // pos / P: the product is short by at most one
        int lp = (int)__umulhi((uint32_t)pos, p.page_inv), slot = pos - lp * p.P;
        if (slot >= p.P) {
            ++lp;
            slot -= p.P;
        }
        const int page = __ldg(trow + lp);
        if (page < 0 || page >= p.n_pages) {
            set_flag(p.flags, kDevBadPage);
            return -1;  // never read
        }
        return (page * p.Hkv + kh) * p.P + slot;
    };
    // K rows g and g + 8 of a chunk: dims 32 c + 8 t .. + 7 of the slice, copy
    // 4 h + c
    const uint32_t ring = smem_addr(&sm.ring[warp][0][0][0][lane]);
    constexpr uint32_t kHalf = 8 * 32 * 16;  // bytes of a stage's K, or V
    auto copy_k = [&](int rows, int stage) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = __shfl_sync(0xffffffffu, rows, g + 8 * h);
            const __nv_bfloat16 *src = p.k_pool + (int64_t)max(r, 0) * D + slice * 128 + 8 * t;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                copy16(ring + stage * 2 * kHalf + (4 * h + c) * 512, src + 32 * c, r >= 0);
        }
        copies_commit();
    };
    // V of a chunk: rows, half a warp to a row; or fragments as K's, rows 2t, 2t +
    // 1, 2t + 8, 2t + 9, dims 64 c + 8 g .. + 7 of the slice, copy 4 c + h
    const int up = lane >> 4, q16 = lane & 15;
    auto copy_v = [&](int rows, int stage) {
        const uint32_t dst = ring + (stage * 2 + 1) * kHalf;
        if constexpr (kMmaPv) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const int r = __shfl_sync(0xffffffffu, rows, 2 * t + (h & 1) + (h >> 1) * 8);
                const __nv_bfloat16 *src = p.v_pool + (int64_t)max(r, 0) * D + slice * 128 + 8 * g;
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    copy16(dst + (4 * c + h) * 512, src + 64 * c, r >= 0);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int r = __shfl_sync(0xffffffffu, rows, 2 * k + up);
                copy16(dst + k * 512, p.v_pool + (int64_t)max(r, 0) * D + slice * 128 + 8 * q16, r >= 0);
            }
        }
        copies_commit();
    };
    const uint4(*const frag)[2][8][32] = sm.ring[warp];

    const int step = C * kTeams;
    int ch = rank * kTeams + team;
    {
        int rows[kStages];
#pragma unroll
        for (int k = 0; k < kStages; ++k)
            rows[k] = lookup(ch + k * step);
#pragma unroll
        for (int k = 0; k < kStages; ++k) {
            copy_k(rows[k], k);
            copy_v(rows[k], k);
        }
    }
    int rows_next = lookup(ch + kStages * step);
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
        for (int e = 0; e < 2; ++e)
            end[y][e] = row_lim(p, len, m0 + 8 * y + 2 * t + e);
    // positions every row of the block sees need no mask
    const int all_end = row_lim(p, len, m0), all_begin = lim - p.window;

    // FMAs: rows 2 k and 2 k + 1, dim 8 q16 + d of the slice, over the positions of
    // the lane's half
    float2 o[kMmaPv ? 1 : R / 2][8];
    // mma.sync: om[4 c + k][y][2 d + e] is dim 64 c + 8 g + 2 k + d of row 8 y + 2 t + e
    float om[kMmaPv ? 8 : 1][NT][4];
#pragma unroll
    for (int k = 0; k < (kMmaPv ? 1 : R / 2); ++k)
#pragma unroll
        for (int d = 0; d < 8; ++d)
            o[k][d] = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < (kMmaPv ? 8 : 1); ++k)
#pragma unroll
        for (int y = 0; y < NT; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                om[k][y][e] = 0.f;
    float mref[NT][2], l[NT][2];
#pragma unroll
    for (int y = 0; y < NT; ++y)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            mref[y][e] = NEG_INF;
            l[y][e] = 0.f;
        }

    int stage = 0;
    for (int it = 0; ch < n_chunks; ch += step, ++it, stage = stage + 1 < kStages ? stage + 1 : 0) {
        // ---- S^T = K Q^T: x[y][2 h + e] is index 16 ch + 8 h + g, row 8 y + 2 t + e
        float x[NT][4];
        copies_wait<2 * kStages - 1>();  // (K and V of each later chunk, this one's V)
        {
            uint4 k[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    k[h][c] = frag[stage][0][4 * h + c][lane];
            // two chains of sums per tile
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
                    x[y][e] = z[y][0][e] + z[y][1][e];
        }
        const int rows = rows_next;      // of the chunk kStages on
        copy_k(rows, stage);
        rows_next = lookup(ch + (kStages + 1) * step);
        if constexpr (kTeam > 1) {
            // sum over the team's slices, in one order for all of its warps
            auto &xs = sm.s[it & 1];
#pragma unroll
            for (int y = 0; y < NT; ++y)
                *reinterpret_cast<float4 *>(&xs[warp][lane][4 * y]) =
                    make_float4(x[y][0], x[y][1], x[y][2], x[y][3]);
            named_barrier(1 + team, 32 * kTeam);
#pragma unroll
            for (int y = 0; y < NT; ++y) {
                float4 a = *reinterpret_cast<const float4 *>(&xs[team * kTeam][lane][4 * y]);
#pragma unroll
                for (int w = 1; w < kTeam; ++w) {
                    const float4 v = *reinterpret_cast<const float4 *>(&xs[team * kTeam + w][lane][4 * y]);
                    a.x += v.x;
                    a.y += v.y;
                    a.z += v.z;
                    a.w += v.w;
                }
                x[y][0] = a.x;
                x[y][1] = a.y;
                x[y][2] = a.z;
                x[y][3] = a.w;
            }
        }
        // ---- masked scores in log2 units; does some row's maximum grow too far?
        const int i0 = ch * kChunk;
        const int p0 = i0 < sink_end ? i0 : i0 + shift;
        const bool one_run = i0 + kChunk <= sink_end || i0 >= sink_end;
        const bool whole = one_run && i0 + kChunk <= n && p0 + kChunk <= all_end &&
                           (p0 >= all_begin || p0 + kChunk <= p.sinks);
        bool grow = false;
#pragma unroll
        for (int y = 0; y < NT; ++y) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v = x[y][e] * p.scale_log2;
                if (!whole) {
                    const int i = i0 + g + 8 * (e >> 1);
                    const int pos = i < sink_end ? i : i + shift;
                    if (i >= n || pos >= end[y][e & 1] ||
                        (pos < end[y][e & 1] - p.window && pos >= p.sinks))
                        v = NEG_INF;
                }
                x[y][e] = v;
                grow = grow || v > mref[y][e & 1] + kRescaleLog2;
            }
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int y = 0; y < NT; ++y) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(x[y][e], x[y][2 + e]);
#pragma unroll
                    for (int k = 4; k < 32; k <<= 1)
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
                    const float m_new = fmaxf(mref[y][e], mx);
                    const float al = mref[y][e] == NEG_INF ? 0.f : fast_exp2(mref[y][e] - m_new);
                    mref[y][e] = m_new;
                    l[y][e] *= al;
                    if constexpr (kMmaPv) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            om[k][y][e] *= al;
                            om[k][y][2 + e] *= al;
                        }
                    } else if (g == 0 && 2 * t + e < R) {
                        sm.alpha[warp][2 * t + e] = al;
                    }
                }
            }
            if constexpr (!kMmaPv) {
                __syncwarp();
#pragma unroll
                for (int k = 0; k < R / 2; ++k) {
                    const float2 al = *reinterpret_cast<const float2 *>(&sm.alpha[warp][2 * k]);
#pragma unroll
                    for (int d = 0; d < 8; ++d)
                        o[k][d] = __fmul2_rn(o[k][d], al);
                }
            }
        }
        // ---- P: by position in shared memory, or in three parts in fragments:
        // part[y][h][f] holds positions 8 h + 2 t and + 1 of row 8 y + g
        uint32_t part[kMmaPv ? NT : 1][2][3];
#pragma unroll
        for (int y = 0; y < NT; ++y) {
            const float n0 = mref[y][0] == NEG_INF ? 0.f : -mref[y][0];
            const float n1 = mref[y][1] == NEG_INF ? 0.f : -mref[y][1];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 pr = make_float2(fast_exp2(x[y][2 * h] + n0), fast_exp2(x[y][2 * h + 1] + n1));
                l[y][0] += pr.x;
                l[y][1] += pr.y;
                if constexpr (kMmaPv) {
                    split3(pr.x, pr.y, part[y][h]);
#pragma unroll
                    for (int f = 0; f < 3; ++f)
                        part[y][h][f] = transpose8(part[y][h][f]);
                } else if (R > 4 || t < 2) {
                    *reinterpret_cast<float2 *>(&sm.p[warp][8 * h + g][2 * t]) = pr;
                }
            }
        }
        // ---- O += P V (rows that were not read are zeros)
        copies_wait<2 * kStages - 1>();
        if constexpr (kMmaPv) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint4 v[4];
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    v[h] = frag[stage][1][4 * c + h][lane];
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
                            mma16816(acc[k][y], a0, a1, a2, a3, part[y][0][f], part[y][1][f]);
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int y = 0; y < NT; ++y)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            om[4 * c + k][y][e] += acc[k][y][e];
            }
        } else {
            __syncwarp();
            const uint4 *const v_rows = &frag[stage][1][0][lane];
#pragma unroll
            for (int i = 0; i < kChunk / 2; ++i) {
                const uint4 w = v_rows[i * 32];
                const float v[8] = {bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y),
                                    bf_lo(w.z), bf_hi(w.z), bf_lo(w.w), bf_hi(w.w)};
#pragma unroll
                for (int k = 0; k < R / 4; ++k) {
                    const float4 pr = *reinterpret_cast<const float4 *>(&sm.p[warp][2 * i + up][4 * k]);
#pragma unroll
                    for (int d = 0; d < 8; ++d) {
                        const float2 vv = make_float2(v[d], v[d]);
                        o[2 * k][d] = __ffma2_rn(make_float2(pr.x, pr.y), vv, o[2 * k][d]);
                        o[2 * k + 1][d] = __ffma2_rn(make_float2(pr.z, pr.w), vv, o[2 * k + 1][d]);
                    }
                }
            }
            __syncwarp();  // (every lane read the chunk's V and P)
        }
        copy_v(rows, stage);
    }

    copies_wait<0>();
    __syncwarp();
    float(*const o_part)[128] = reinterpret_cast<float(*)[128]>(&sm.ring[warp][0][0][0][0]);
    // ---- join: O by warp, maxima and sums by team --------------------------------
#pragma unroll
    for (int y = 0; y < NT; ++y) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int k = 4; k < 32; k <<= 1)
                l[y][e] += __shfl_xor_sync(0xffffffffu, l[y][e], k);
            const int r = 8 * y + 2 * t + e;
            if (slice == 0 && g == 0 && r < R) {
                sm.m[team][r] = mref[y][e];
                sm.l[team][r] = l[y][e];
            }
        }
    }
    if constexpr (kMmaPv) {
#pragma unroll
        for (int y = 0; y < NT; ++y)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int k = 0; k < 4; k += 2)
                        *reinterpret_cast<float4 *>(&o_part[8 * y + 2 * t + e][64 * c + 8 * g + 2 * k]) =
                            make_float4(om[4 * c + k][y][e], om[4 * c + k][y][2 + e], om[4 * c + k + 1][y][e],
                                        om[4 * c + k + 1][y][2 + e]);
    } else {
        // the lower half of the warp ends up with the even rows, the upper with the odd
#pragma unroll
        for (int k = 0; k < R / 2; ++k) {
            float sum[8];
#pragma unroll
            for (int d = 0; d < 8; ++d)
                sum[d] = (up ? o[k][d].y : o[k][d].x) +
                         __shfl_xor_sync(0xffffffffu, up ? o[k][d].x : o[k][d].y, 16);
            float4 *dst = reinterpret_cast<float4 *>(&o_part[2 * k + up][8 * q16]);
            dst[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
            dst[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
        }
    }
    cluster_sync();
    const uint32_t m_addr = smem_addr(sm.m), l_addr = smem_addr(sm.l), o_addr = smem_addr(sm.ring);
    for (int e = rank * kWinThreads + threadIdx.x; e < n_rows * (D / 4); e += C * kWinThreads) {
        const int r = e / (D / 4), d = e % (D / 4) * 4;
        float top = NEG_INF;
        for (int k = 0; k < C; ++k)
#pragma unroll
            for (int w = 0; w < kTeams; ++w)
                top = fmaxf(top, peer_f32(peer_addr(m_addr, k) + (w * R + r) * 4));
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
        for (int k = 0; k < C; ++k) {
#pragma unroll
            for (int w = 0; w < kTeams; ++w) {
                const uint32_t at = (w * R + r) * 4;
                // (a team without positions: 2^-inf = 0)
                const float wt = fast_exp2(peer_f32(peer_addr(m_addr, k) + at) - top);
                sum = fmaf(wt, peer_f32(peer_addr(l_addr, k) + at), sum);
                const float4 v = peer_f32x4(peer_addr(o_addr, k) +
                                            (uint32_t)((w * kTeam + d / 128) * sizeof(sm.ring[0])) +
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
template <int D, int R>
int win_clusters(int C)
{
    static std::atomic<int> known[kMaxDevices][kMaxCluster + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return 0;
    int n = known[dev][C].load(std::memory_order_relaxed);
    if (n == 0) {
        constexpr size_t bytes = sizeof(WinSmem<D, R>);
        static std::atomic<bool> configured[kMaxDevices];
        if (set_smem_limit_once(attn_win_kernel<D, R>, bytes, configured) != cudaSuccess)
            return 0;
        WinLaunch launch(C, C, bytes, nullptr);
        launch.cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, attn_win_kernel<D, R>, &launch.cfg) != cudaSuccess)
            return 0;
        known[dev][C].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <int D, int R>
cudaError_t launch_win(const WinParams &p, int grid, cudaStream_t stream)
{
    constexpr size_t bytes = sizeof(WinSmem<D, R>);
    static_assert(win_blocks(R) * (bytes + 1024) <= 228 * 1024, "shared memory");
    static std::atomic<bool> configured[kMaxDevices];
    const cudaError_t e = set_smem_limit_once(attn_win_kernel<D, R>, bytes, configured);
    if (e != cudaSuccess)
        return e;
    WinLaunch launch(p.whole, grid, bytes, stream);
    return cudaLaunchKernelEx(&launch.cfg, attn_win_kernel<D, R>, p);
}

template <int R>
cudaError_t launch_win_rows(const WinParams &p, int grid, cudaStream_t stream)
{
    return p.D == 128   ? launch_win<128, R>(p, grid, stream)
           : p.D == 256 ? launch_win<256, R>(p, grid, stream)
                        : launch_win<512, R>(p, grid, stream);
}

template <int R>
int win_clusters_rows(int D, int C)
{
    return D == 128 ? win_clusters<128, R>(C) : D == 256 ? win_clusters<256, R>(C) : win_clusters<512, R>(C);
}

}  // namespace

// Blocks per cluster, and what the call then costs (in chunks).  The blocks of
// one wave run side by side; a block's time is its warps' chunks one after
// another, plus starting and joining (about kEntry chunks).  So: the cluster
// size whose waves times that is least (ties to the smaller).
WinSplit win_split(const WinParams &p, int64_t units)
{
    constexpr int kEntry = 4;
    // (a block's rows span at most so many of the call's)
    const int span = std::min(p.W, (p.RB + p.G - 2) / p.G + 1);
    const int64_t seen = std::min<int64_t>(p.max_len, (int64_t)p.window + p.sinks + span);
    const int64_t chunks = (seen + kChunk - 1) / kChunk;
    const int teams = kWinWarps / (p.D / 128);
    WinSplit best = {1, INT64_MAX};
    for (int C = 1; C <= kMaxCluster; ++C) {
        const int64_t at_once = p.RB == 4   ? win_clusters_rows<4>(p.D, C)
                                : p.RB == 8 ? win_clusters_rows<8>(p.D, C)
                                            : win_clusters_rows<16>(p.D, C);
        if (at_once <= 0)
            continue;
        const int64_t waves = (units + at_once - 1) / at_once;
        const int64_t cost = waves * ((chunks + C * teams - 1) / (C * teams) + kEntry);
        if (cost < best.cost)
            best = {C, cost};
    }
    return best;
}

cudaError_t launch_attn_win(const WinParams &p, int grid, cudaStream_t stream)
{
    return p.RB == 4   ? launch_win_rows<4>(p, grid, stream)
           : p.RB == 8 ? launch_win_rows<8>(p, grid, stream)
                       : launch_win_rows<16>(p, grid, stream);
}

}  // namespace tfp
