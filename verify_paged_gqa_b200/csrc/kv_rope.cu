// kv_rope.cu -- the row write with rotary positions of several axes.
//
// TensorFold #1620, opening comment, "Writes": a step's new K and V rows are
// copied into the stream's pages.  Here the query and key rows of the step
// are turned by their rotary positions on the way: pair i of a head's first
// rotary_dim dims, (a, b), becomes
//     a' = a cos t - b sin t,   b' = b cos t + a sin t,
//     t  = position[axis(i)] * inv_freq[i],
// with one position per axis (time, height, width of an image token; one axis
// is the usual text position).  The turned keys and the values go to page
// table[s][pos / P], slot pos % P, the turned queries to a buffer of their own
// (or back in place).
//
// The angle is formed in 64 bits and reduced to half turns there (a position
// of 10^6 leaves an fp32 angle 0.06 radians off), its sine and cosine are
// fp32, the products fp32, and each output is rounded once, to bf16.
//
// Memory bound: every input row is read once and every output written once.
// The row's rotary_dim / 2 angles are computed once, into shared memory, and
// serve all its heads; a thread moves 32 bytes (two 16-byte vectors: 8 pairs)
// at a time, and the first loads are issued before the angles are formed.
#include "launch.cuh"

#include <algorithm>

namespace tfp {

namespace {

constexpr int kRopeThreads = 256;
constexpr int64_t kWarpRows = 4096;  // from so many rows on, one warp per row

// The row's K/V destination (element offset of KV head 0), or -1: skipped.
__device__ __forceinline__ int64_t row_slot(const RopeParams &p, int s, int r)
{
    const int len = __ldg(p.lens + s);
    if (len < p.W || len > p.max_len || (int64_t)len > (int64_t)p.table_stride * p.P)
        return -1;
    const int pos = len - p.W + r;
    const int lp = pos / p.P;
    const int page = __ldg(p.table + (int64_t)s * p.table_stride + lp);
    if (page < 0 || page >= p.n_pages)
        return -1;
    return ((int64_t)page * p.Hkv * p.P + (pos - lp * p.P)) * p.D;
}

// cos and sin of pair i's angle at this row.
__device__ __forceinline__ float2 pair_turn(const RopeParams &p, const int32_t *position, int i)
{
    // half turns in [-1, 1]
    double x = (double)__ldg(position + p.pair_axis[i]) * (double)__ldg(p.inv_freq + i) *
               0.31830988618379067154;  // 1 / pi
    x -= 2.0 * rint(0.5 * x);
    float2 t;
    sincospif((float)x, &t.y, &t.x);
    return t;
}

// (a, b) packed low / high turned by t and rounded.
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}

__device__ __forceinline__ float turn_a(float a, float b, float2 t) { return fmaf(a, t.x, -(b * t.y)); }
__device__ __forceinline__ float turn_b(float a, float b, float2 t) { return fmaf(b, t.x, a * t.y); }

// Pairs (a_j, b_j) of two vectors of 8 dims (j = 0 .. 7), angles t[0 .. 7].
__device__ __forceinline__ void turn_halves(uint4 &a, uint4 &b, const float2 *t)
{
    uint32_t *aw = &a.x, *bw = &b.x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float4 tt = *reinterpret_cast<const float4 *>(t + 2 * e);  // two pairs
        const float2 t0 = make_float2(tt.x, tt.y), t1 = make_float2(tt.z, tt.w);
        const float a0 = bf_lo(aw[e]), a1 = bf_hi(aw[e]), b0 = bf_lo(bw[e]), b1 = bf_hi(bw[e]);
        aw[e] = pack2(turn_a(a0, b0, t0), turn_a(a1, b1, t1));
        bw[e] = pack2(turn_b(a0, b0, t0), turn_b(a1, b1, t1));
    }
}

// Pairs of neighbouring dims of one vector of 8 dims, angles t[0 .. 3].
__device__ __forceinline__ void turn_adjacent(uint4 &a, const float2 *t)
{
    uint32_t *aw = &a.x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float x = bf_lo(aw[e]), y = bf_hi(aw[e]);
        aw[e] = pack2(turn_a(x, y, t[e]), turn_b(x, y, t[e]));
    }
}

// Where item `it` of a row lies: 32 bytes of a query head, a key head or a
// value head, in this order.  `shift`: log2 of a head's items.
struct Item {
    int kind, h, c;  // 0: query, 1: key, 2: value; the head; its item
    bool turned;
    int d0, d1;      // first dims of its two vectors of 8
};

__device__ __forceinline__ Item item_of(const RopeParams &p, int it, int shift, int half)
{
    const int q_items = p.Hq << shift, k_items = p.Hkv << shift;
    Item x;
    x.kind = it < q_items ? 0 : it < q_items + k_items ? 1 : 2;
    const int y = it - (x.kind == 0 ? 0 : x.kind == 1 ? q_items : q_items + k_items);
    x.h = y >> shift;
    x.c = y & ((1 << shift) - 1);
    // dims (8c, half + 8c) of a turned half split, else 16 dims in a row
    x.turned = x.kind != 2 && 8 * x.c < half;
    x.d0 = x.turned && !p.adjacent ? 8 * x.c : 16 * x.c;
    x.d1 = x.turned && !p.adjacent ? half + 8 * x.c : 16 * x.c + 8;
    return x;
}

// rotary_dim a multiple of 16: whole vectors are turned or kept.  kGroup
// threads take a row: a block's 256 while there are few rows, a warp once the
// rows alone fill the GPU (no barriers then).  4,096 rows of 4 streams, 48
// heads of 128 dims: 72 us by warps (5,560 GB/s), 84 by blocks.
template <int kThreads, int kGroup>
__global__ void __launch_bounds__(kThreads) kv_rope_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int kGroups = kThreads / kGroup;
    constexpr int kBatch = 2;  // items a thread has in flight
    allow_dependent_launch();  // the attention kernel after it may be scheduled now
    __shared__ __align__(16) float2 turns[kGroups][256];
    __shared__ int64_t slots[kGroups];
    const int group = threadIdx.x / kGroup, lane = threadIdx.x % kGroup;
    float2 *turn = turns[group];
    const int half = p.rotary / 2;
    const int shift = 31 - __clz(p.D / 16);
    const int n = (p.Hq + 2 * p.Hkv) << shift;
    auto sync = [] {
        if constexpr (kGroup == 32)
            __syncwarp();
        else
            __syncthreads();
    };
    const int64_t rows = (int64_t)p.S * p.W;
    for (int64_t row = (int64_t)blockIdx.x * kGroups + group; row < rows; row += (int64_t)gridDim.x * kGroups) {
        const __nv_bfloat16 *qs = p.q + row * p.q_stride, *ks = p.k + row * p.k_stride,
                            *vs = p.v + row * p.v_stride;
        __nv_bfloat16 *qd = p.q_out + row * p.Hq * p.D;
        const int64_t head_step = (int64_t)p.P * p.D;  // between a slot's KV heads
        int64_t slot = -1;
        for (int base = 0; base < n; base += kBatch * kGroup) {
            uint4 a[kBatch], b[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int it = base + k * kGroup + lane;
                if (it < n) {
                    const Item x = item_of(p, it, shift, half);
                    const __nv_bfloat16 *src = (x.kind == 0 ? qs : x.kind == 1 ? ks : vs) + x.h * p.D;
                    // (not __ldg: q may be its own output)
                    a[k] = *reinterpret_cast<const uint4 *>(src + x.d0);
                    b[k] = *reinterpret_cast<const uint4 *>(src + x.d1);
                }
            }
            if (base == 0) {
                // the row's angles and slot, while its first items are on their way
                sync();  // (the previous row's are no longer read)
                if (lane == kGroup - 1) {
                    const int s = static_cast<int>(row / p.W);
                    slots[group] = row_slot(p, s, static_cast<int>(row - (int64_t)s * p.W));
                }
                for (int i = lane; i < half; i += kGroup)
                    turn[i] = pair_turn(p, p.positions + row * p.n_axes, i);
                sync();
                slot = slots[group];
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int it = base + k * kGroup + lane;
                if (it >= n)
                    continue;
                const Item x = item_of(p, it, shift, half);
                if (x.kind != 0 && slot < 0)
                    continue;
                if (x.turned) {
                    if (p.adjacent) {
                        turn_adjacent(a[k], turn + 8 * x.c);
                        turn_adjacent(b[k], turn + 8 * x.c + 4);
                    } else {
                        turn_halves(a[k], b[k], turn + 8 * x.c);
                    }
                }
                __nv_bfloat16 *dst = x.kind == 0 ? qd + x.h * p.D
                                                 : (x.kind == 1 ? p.k_pool : p.v_pool) + slot + x.h * head_step;
                *reinterpret_cast<uint4 *>(dst + x.d0) = a[k];
                *reinterpret_cast<uint4 *>(dst + x.d1) = b[k];
            }
        }
    }
}

// Any other rotary_dim: one block per row, whose warps take a head each
// through shared memory, dim by dim (every read comes before the row's
// writes, so q may be turned in place).  4,096 rows of 4 streams, 48 heads of 128
// dims: 213 us at rotary_dim 90, where whole vectors take 75 (87 in adjacent
// pairs); 64 rows 10 us and 8.
__global__ void __launch_bounds__(kRopeThreads) kv_rope_odd_kernel(const __grid_constant__ RopeParams p)
{
    allow_dependent_launch();
    __shared__ __align__(16) float2 turn[256];
    __shared__ int64_t slot_sh;
    __shared__ __align__(16) uint32_t stage[kRopeThreads / 32][256];
    const int half = p.rotary / 2;
    const int64_t rows = (int64_t)p.S * p.W;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        __syncthreads();  // the previous row's angles are no longer read
        if (threadIdx.x == kRopeThreads - 1) {
            const int s = static_cast<int>(row / p.W);
            slot_sh = row_slot(p, s, static_cast<int>(row - (int64_t)s * p.W));
        }
        for (int i = threadIdx.x; i < half; i += kRopeThreads)
            turn[i] = pair_turn(p, p.positions + row * p.n_axes, i);
        __syncthreads();
        const int64_t slot = slot_sh;
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        const int heads = p.Hq + (slot >= 0 ? 2 * p.Hkv : 0);
        for (int h = warp; h < heads; h += kRopeThreads / 32) {
            const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hkv;
            const int hk = h - p.Hq - (is_k ? 0 : p.Hkv);
            const __nv_bfloat16 *src = is_q   ? p.q + row * p.q_stride + (int64_t)h * p.D
                                       : is_k ? p.k + row * p.k_stride + (int64_t)hk * p.D
                                              : p.v + row * p.v_stride + (int64_t)hk * p.D;
            __nv_bfloat16 *dst = is_q ? p.q_out + (row * p.Hq + h) * p.D
                                      : (is_k ? p.k_pool : p.v_pool) + slot + (int64_t)hk * p.P * p.D;
            for (int w = lane; w < p.D / 2; w += 32)
                stage[warp][w] = reinterpret_cast<const uint32_t *>(src)[w];
            __syncwarp();
            auto at = [&](int d) { return d & 1 ? bf_hi(stage[warp][d >> 1]) : bf_lo(stage[warp][d >> 1]); };
            // the turned value of dim d < rotary
            auto value = [&](int d) {
                const bool second = p.adjacent ? (d & 1) != 0 : d >= half;
                const int i = p.adjacent ? d >> 1 : second ? d - half : d;
                const float2 t = turn[i];
                const int other = p.adjacent ? d ^ 1 : second ? d - half : d + half;
                return second ? turn_b(at(other), at(d), t) : turn_a(at(d), at(other), t);
            };
            for (int w = lane; w < p.D / 2; w += 32) {
                const int d = 2 * w;  // rotary is even: both dims are turned, or neither
                uint32_t word = stage[warp][w];
                if ((is_q || is_k) && d < p.rotary)
                    word = pack2(value(d), value(d + 1));
                reinterpret_cast<uint32_t *>(dst)[w] = word;
            }
            __syncwarp();
        }
    }
}

}  // namespace

cudaError_t launch_kv_rope(const RopeParams &p, cudaStream_t stream)
{
    const int64_t rows = (int64_t)p.S * p.W;
    if (rows == 0)
        return cudaSuccess;
    const int64_t most = 0x7fffffff;
    if (p.rotary % 16 != 0) {
        kv_rope_odd_kernel<<<static_cast<unsigned>(std::min(rows, most)), kRopeThreads, 0, stream>>>(p);
    } else if (rows < kWarpRows) {
        kv_rope_kernel<kRopeThreads, kRopeThreads><<<static_cast<unsigned>(rows), kRopeThreads, 0, stream>>>(p);
    } else {
        constexpr int threads = 128, per_block = threads / 32;
        kv_rope_kernel<threads, 32><<<static_cast<unsigned>(std::min((rows + per_block - 1) / per_block, most)),
                                      threads, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace tfp
