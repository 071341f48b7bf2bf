// tf_paged.cu -- the C ABI: argument checks, the launch plan, dispatch.
//
// Every entry point checks its host arguments before enqueueing anything
// and returns a TF_* status.  The plan (row blocks, context chunk, grid)
// depends only on host arguments and the device's SM count, so a captured
// graph stays valid while lens grow up to max_len.
#include "../../include/tf_paged.h"
#include "../../include/tf_paged_testing.h"
#include "launch.cuh"
#include "plan.cuh"

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

namespace tfp {
namespace {

// The SM count of the current device, queried once per device.  Host threads
// making their first calls at once may each query it and store the same
// value; the atomics keep that race well defined.
int device_sm_count(int *sms)
{
    static std::atomic<int> cached[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return TF_ECUDA;
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            n <= 0)
            return TF_ECUDA;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    *sms = n;
    return TF_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int check_pool_streams(const tf_kv_pool *pool, const tf_streams *st)
{
    if (!pool || !st)
        return TF_EINVAL;
    if (pool->n_pages < 1 || pool->n_kv_heads < 1 || pool->page_size < 1)
        return TF_EINVAL;
    if (pool->head_dim != 128 && pool->head_dim != 256 && pool->head_dim != 512)
        return TF_EUNSUPPORTED;
    if (st->n_streams < 0 || st->table_stride < 1 || st->max_len < 1)
        return TF_EINVAL;
    if ((int64_t)st->max_len > (int64_t)st->table_stride * pool->page_size)
        return TF_EINVAL;
    if ((int64_t)st->n_streams * st->table_stride > INT32_MAX)
        return TF_EINVAL;
    if (st->n_streams > 0 && (!st->table || !st->lens || !aligned4(st->table) || !aligned4(st->lens)))
        return TF_EINVAL;
    if (!pool->k_pool || !pool->v_pool || !aligned16(pool->k_pool) || !aligned16(pool->v_pool))
        return TF_EINVAL;
    return TF_OK;
}

enum class Kernel { kSimt, kPrompt, kPm, kWin };

// Workspace: the 256-byte header (status word, wait site, the launch's tile
// count at byte 64), each stream's first tile (int64), then two partial slots
// per CTA of min(RB, M) rows x (D + 2) floats (rounded up to 16 bytes).
constexpr size_t kWsTotalOffset = 64;

size_t ws_part_offset(int S)
{
    return kWsHeaderBytes + (((size_t)S * 8 + 255) / 256) * 256;
}

// What every attention call of at most p.S streams and p.M rows per (stream, KV
// head) fits into, whichever kernel it takes and however short it is: two slots
// for each of `cap` CTAs, of as many rows as a row block of the head dim can
// have.  It grows with S and M and depends on nothing else of the call, so the
// figure for the largest shape serves the smaller ones.
size_t ws_bytes_of_any(AttnParams p, int cap)
{
    p.SR = std::min(p.M, p.D == 128 ? prompt_rows() : kPmWideRows);
    return ws_part_offset(p.S) + (size_t)2 * cap * part_slot_floats(p) * sizeof(float);
}

// Entry tiles per unit (plan.cuh), measured: at head dim 512 a unit start
// costs about 8 tiles' worth of streaming (the ring holds less than one
// tile, so the pipeline drains and refills); the prompt kernel's split
// units (more than 64 rows per KV head over long contexts) pay its serial
// epilogue and its query load, about 8 of its tiles; the CUDA-core decode
// kernel's segment starts overlap with its deep ring and cost nothing
// measurable.
constexpr int kEntryPm512 = 8;
constexpr int kEntryPm128 = 6;
constexpr int kEntryPrompt = 8;
constexpr int kEntrySimt = 0;

// Decode blocks at head dim 128 take the position-major kernel from this
// max_len on (measured crossover near 5,700 positions).
constexpr int kPmDecodeMinLen = 6144;

// A sliding-window call's host arguments.  `kernel` (tests only): 0 the
// library's choice, 1 the tensor-core kernels, 2 the cluster kernel.
struct Window {
    int32_t window = 0;
    int32_t sinks = 0;
    int32_t kernel = 0;
};

struct Plan {
    WinParams p;  // a plain call launches its AttnParams part
    int grid;
    size_t ws_bytes;  // this call's need
    size_t ws_any;    // that of any call of its size or less
    Kernel kernel;  // which partial kernel runs the call
};

bool pool_rows_past_31_bits(const tf_kv_pool *pool)
{
    return (int64_t)pool->n_pages * pool->n_kv_heads * pool->page_size > INT32_MAX;
}

// How many pieces a sliding-window call on the tensor-core kernels cuts each
// unit into, one to a CTA (plan.cuh); 0: the work is dealt out evenly.  Dealing
// out costs every CTA a second start, a walk over all row blocks at both ends
// and a merge that looks at every row.  So units that fit the CTAs are cut into
// as many pieces as there are CTAs for (8 units of seven row blocks over 4,096
// positions: 53 us, dealt out 59, whole 72), and more units stay whole (2
// streams x 4,096 rows of 32 heads over 4,096 positions: 925 us, dealt out
// 1,128; over 1,024: 419 and 608), unless the last round would leave more than
// kIdle tiles per unit to idle CTAs (64 rows over 4,096 positions at head dim
// 128: 240 units, 8 idle tiles, 147 us and dealt out 176; 160 units, 28 idle
// tiles, 145 and 119).  Head dims 256 and 512 have longer tiles.  `tiles`: of a
// unit at most.
int32_t window_pieces(int32_t head_dim, int64_t units, int64_t cap, int64_t tiles)
{
    const int64_t kIdle = head_dim == 128 ? 12 : head_dim == 256 ? 4 : 2;
    if (units == 0 || units > INT32_MAX / 2)
        return 0;
    if (units <= cap)
        return static_cast<int32_t>(std::min<int64_t>(cap / units, tiles));
    const int64_t idle = (units + cap - 1) / cap * cap - units;
    return idle * tiles <= kIdle * units;
}

// Row blocks of the position-major or prompt kernel against the cluster kernel
// (attn_win.cu) for a sliding-window call, by estimates fitted to both kernels
// over 638 calls (head dims 128, 256 and 512; 8 to 1,600 rows per KV head; 2 to
// 256 units; windows of 64 to 8,192): the choice is 0.6% slower than the faster
// of the two in the geometric mean, 28% at worst, where always the cluster
// kernel up to 16 rows was 11%, never 25%.  Over 400 others, drawn over all page
// sizes and ratios of heads, it was 0.5%; at worst 55% (1,540 rows at head dim 512
// over pages of 16: 888 us, 574 on the cluster kernel), 46% (7 rows at head dim
// 256 over pages of 16) and 35% (one row of 3 streams at head dim 512 over pages
// of 512: 30.5 us and 22.7).  In tenths of microseconds, without what both take to
// start:
//   cluster      its chunks one after another, 1.2 to 2.1 us each: it reads the
//                unit again for every 16 rows, and its products run on mma.sync
//                and FMAs
//   tensor core  5 to 9 us more to start, then 1.4, 3.3 or 5 us per 128-position
//                tile that a CTA takes (twice that over pages below 32 positions
//                at head dims 256 and 512: copies by the piece), 11 to 13 per
//                unit, and 20 where the work is dealt out
// Sets p.RB and p.whole for the cluster kernel when it is taken.
bool takes_win_kernel(WinParams &p, int sms, int forced)
{
    const int d = p.D == 128 ? 0 : p.D == 256 ? 1 : 2;
    WinParams c = p;
    c.RB = p.M <= 4 ? 4 : p.M <= 8 ? 8 : 16;
    const int64_t heads = (int64_t)p.S * p.Hkv;
    const int64_t units = heads * ((p.M + c.RB - 1) / c.RB);
    if (units > INT32_MAX / kMaxCluster)
        return false;
    constexpr int kChunk4 = 12, kChunk8[3] = {12, 17, 15}, kChunk16[3] = {17, 21, 20};
    const WinSplit split = win_split(c, units);
    const int64_t cluster =
        split.cost < INT64_MAX / 64
            ? split.cost * (c.RB == 4 ? kChunk4 : c.RB == 8 ? kChunk8[d] : kChunk16[d])
            : INT64_MAX;
    const int rows = p.D > 128 || p.M <= 32 ? 32 : p.M <= 64 ? 64 : 128;  // of its row blocks
    const int64_t blocks = heads * ((p.M + rows - 1) / rows);
    const int64_t seen = std::min<int64_t>(p.max_len, (int64_t)p.window + p.sinks + std::min(p.W, (rows + p.G - 1) / p.G));
    const int64_t tiles2 = 2 * ((seen + 127) / 128) + 1;  // (half a tile more for the edges)
    constexpr int kStart[3] = {80, 50, 90}, kTile[3] = {14, 33, 50}, kUnit[3] = {130, 110, 130};
    const int64_t tile = p.P < 32 && p.D > 128 ? 2 * kTile[d] : kTile[d];
    constexpr int kDealt = 200;
    const int64_t pieces = window_pieces(p.D, blocks, sms, (tiles2 + 1) / 2);
    int64_t tensor = kStart[d];
    if (pieces == 0)
        tensor += kDealt + blocks * (tiles2 * tile / 2 + kUnit[d]) / sms;
    else if (pieces > 1)
        tensor += ((tiles2 + 1) / 2 + pieces - 1) / pieces * tile + kUnit[d];
    else
        tensor += (blocks + sms - 1) / sms * (tiles2 * tile / 2 + kUnit[d]);
    if (forced == 1 || (forced == 0 && cluster >= tensor))
        return false;
    p.RB = c.RB;
    p.whole = split.C;
    return true;
}

int make_plan(const tf_kv_pool *pool, const tf_streams *st, int32_t Hq, int32_t rows,
              int32_t rows_max, bool tree, Plan *plan, float scale = 1.f, const Window *win = nullptr)
{
    int rc = check_pool_streams(pool, st);
    if (rc != TF_OK)
        return rc;
    if (Hq < 1 || Hq % pool->n_kv_heads != 0)
        return TF_EINVAL;
    if (rows < 1 || rows > rows_max || st->max_len < rows)
        return TF_EINVAL;
    const int G = Hq / pool->n_kv_heads;
    const int64_t M = (int64_t)G * rows;
    if (M > (1 << 20))
        return TF_EINVAL;
    if (win && (win->window < 1 || win->sinks < 0))
        return TF_EINVAL;
    WinParams &p = plan->p;
    p = WinParams{};
    p.P = pool->page_size;
    if (win) {
        // a window or sinks past every length see what max_len does
        p.page_inv = p.P == 1 ? UINT32_MAX : (uint32_t)((1ull << 32) / p.P);
        p.window = win->window < st->max_len ? win->window : st->max_len;
        p.sinks = win->sinks < st->max_len ? win->sinks : st->max_len;
    }
    p.n_pages = pool->n_pages;
    p.Hkv = pool->n_kv_heads;
    p.D = pool->head_dim;
    p.table_stride = st->table_stride;
    p.S = st->n_streams;
    p.max_len = st->max_len;
    p.Hq = Hq;
    p.G = G;
    p.W = rows;
    p.M = static_cast<int32_t>(M);
    p.has_tree = tree ? 1 : 0;
    p.withhold = 0;
    p.wait_limit = kWaitLimitCycles;
    // Rows sharing a KV head go to the tensor cores as a dense QK^T / PV
    // tile: up to 64 rows (any count at head dims 256 and 512, in blocks of
    // 32) with the positions on the MMA's M, larger blocks with the rows
    // there.  At head dim 128 that holds for a single CUDA-core row block
    // too (decode at GQA 4): its two MMA issuers keep pace with HBM at any
    // clock, where the CUDA-core kernel's FMAs fall behind under the power
    // cap (12 x 40,960 decode: 341 -> 296 us per call).  Head dim 512 keeps
    // such calls on the CUDA-core kernel.  Pages that are not a multiple of
    // 128 positions: the tensor-core kernels assemble each tile from page
    // pieces, one TMA box per set bit of a piece's length, so small pages
    // cost many box loads per tile.  For a single 4-row block (decode at
    // GQA <= 4) the CUDA-core kernel, which copies pieces into its own
    // smaller tiles, is then faster below 128 positions unless the page is a
    // multiple of 64 (12 x 40,960 decode, GB/s, CUDA-core / tensor-core:
    // pages of 37 3,378 / 1,915; 48 3,995 / 3,175; 64 5,045 / 5,190; 96
    // 5,368 / 4,830; 100 4,208 / 3,599; 200 4,555 / 4,951; 509 4,697 /
    // 5,527).  Several row blocks would each re-read the K/V on the CUDA-core
    // kernel, so larger blocks always take the tensor cores (verify
    // 4 x 131,072 in pages of 64: 311 against 4,467 GB/s).  Pools past 2^31
    // rows run on the CUDA-core kernel.
    const bool small_odd_pages = p.P < 128 && p.P % 64 != 0;
    // A decode block also stays on the CUDA-core kernel for short contexts:
    // the position-major kernel pays about six tiles (768 positions) to start
    // each (stream, KV head) unit, which outweighs its steady-state lead
    // below about 6,000 positions (GB/s, position-major / CUDA-core: 64 x
    // 2,048 4,507 / 5,112; 256 x 512 3,207 / 3,638; 12 x 8,192 5,315 /
    // 5,187; 12 x 40,960 6,875 / 6,061).  max_len bounds every stream, so the
    // choice depends on host arguments only.
    const bool long_context = st->max_len >= kPmDecodeMinLen;
    // The prompt kernel knows no tree masks, and takes positive scales only: it
    // masks raw scores.  Blocks of 64 rows on the position-major kernel do both
    // (the signs in its queries' loads, which the prompt kernel would take at its
    // registers' limit, cost every call of it 0.7 to 2.2%).
    const bool pm_only = tree || !(scale > 0.f);
    plan->kernel = Kernel::kSimt;
    p.RB = kSimtRows;
    if (win) {
        // a sliding window; pools past 2^31 rows are refused
        const int nr = pm_rows(p, pm_only);
        if (pool_rows_past_31_bits(pool))
            return TF_EUNSUPPORTED;
        int sms = 0;
        rc = device_sm_count(&sms);
        if (rc != TF_OK)
            return rc;
        if (takes_win_kernel(p, sms, win->kernel)) {
            plan->kernel = Kernel::kWin;
        } else if (nr > 0) {
            plan->kernel = Kernel::kPm;
            p.RB = nr;
        } else if (prompt_supported(p)) {
            plan->kernel = Kernel::kPrompt;
            p.RB = prompt_rows();
        } else {
            return TF_EUNSUPPORTED;
        }
    } else if (tree) {
        // tree masks: the position-major kernel (any row count), else the
        // CUDA-core kernel (pools past 2^31 rows)
        const int nr = pm_rows(p, pm_only);
        if (nr > 0) {
            plan->kernel = Kernel::kPm;
            p.RB = nr;
        } else if (p.D == 256) {
            return TF_EUNSUPPORTED;
        }
    } else if (p.D == 256) {
        // head dim 256 runs on the position-major kernel only (any row count)
        const int nr = pm_rows(p, pm_only);
        if (nr == 0)
            return TF_EUNSUPPORTED;
        plan->kernel = Kernel::kPm;
        p.RB = nr;
    } else if (M > kSimtRows || (p.D == 128 && !small_odd_pages && long_context)) {
        const int nr = pm_rows(p, pm_only);
        if (nr > 0) {
            plan->kernel = Kernel::kPm;
            p.RB = nr;
        } else if (prompt_supported(p)) {
            plan->kernel = Kernel::kPrompt;
            p.RB = prompt_rows();
        }
    }
    int sms = 0;
    rc = device_sm_count(&sms);
    if (rc != TF_OK)
        return rc;
    p.n_rblk = static_cast<int32_t>((M + p.RB - 1) / p.RB);
    p.SR = static_cast<int32_t>(M < p.RB ? M : p.RB);

    // Entry cost of a unit, in tiles: what starting one more unit costs a
    // CTA relative to streaming one tile of it (measured per kernel).
    p.VT = plan->kernel == Kernel::kPm ? (p.D == 512 ? kEntryPm512 : kEntryPm128)
         : plan->kernel == Kernel::kPrompt ? kEntryPrompt : kEntrySimt;
    // One persistent CTA per SM, but no more than the work the call can have
    // with every stream at max_len (the device splits the actual work).
    const int64_t head_max = win ? head_work(p, st->max_len)
                                 : head_work(static_cast<const AttnParams &>(p), st->max_len);
    const int64_t tiles_max = (int64_t)p.S * p.Hkv * head_max;
    int64_t grid = sms < kMaxCtas ? sms : kMaxCtas;
    if (tiles_max < grid)
        grid = tiles_max > 0 ? tiles_max : 1;
    // A tensor-bound prompt call whose units fill most CTAs (but no more)
    // gives each CTA one whole unit: the split's partials and merge cost more
    // than a few idle SMs (measured on the chunked prompt: 128 units on 148).
    const int64_t units = (int64_t)p.S * p.Hkv * p.n_rblk;
    const int cap = sms < kMaxCtas ? sms : kMaxCtas;
    if (win && plan->kernel != Kernel::kWin)
        p.whole = window_pieces(p.D, units, cap, head_work(p, st->max_len) / p.n_rblk - p.VT + 1);
    else if (plan->kernel == Kernel::kPrompt)
        p.whole = units <= cap && 4 * units >= 3 * (int64_t)cap;
    if (p.whole && plan->kernel != Kernel::kWin)
        grid = std::min<int64_t>(units * p.whole, cap);
    plan->grid = static_cast<int>(plan->kernel == Kernel::kWin ? units * p.whole : grid);
    p.n_cta = plan->grid;
    plan->ws_any = ws_bytes_of_any(p, cap);
    // (a window's kernel is chosen by estimates: its calls ask for ws_any)
    plan->ws_bytes = win ? plan->ws_any
                         : ws_part_offset(p.S) + (size_t)2 * plan->grid * part_slot_floats(p) * sizeof(float);
    return TF_OK;
}

// The test hooks of one call (tf_testing_paged_attn); none in library calls.
struct Faults {
    long long wait_limit = kWaitLimitCycles;
    int32_t withhold = 0;
};

template <class P>
cudaError_t launch_merge(const P &p, cudaStream_t s)
{
    return p.D == 128   ? launch_attn_merge<128>(p, s)
           : p.D == 256 ? launch_attn_merge<256>(p, s)
                        : launch_attn_merge<512>(p, s);
}

// The partial kernel and the merge of a call on the tensor-core kernels.
template <class P>
cudaError_t launch_tensor_core(const P &p, const Plan &plan, cudaStream_t s)
{
    cudaError_t e = plan.kernel == Kernel::kPm ? launch_attn_pm(p, plan.grid, s)
                                               : launch_attn_prompt(p, plan.grid, s);
    return e == cudaSuccess ? launch_merge(p, s) : e;
}

int attn_call(const tf_kv_pool *pool, const tf_streams *st, const void *q, int32_t Hq,
              int32_t rows, int32_t rows_max, const uint8_t *tree, float scale, float *out,
              void *ws, size_t ws_bytes, void *stream, const Faults &faults = Faults{},
              const Window *win = nullptr)
{
    Plan plan;
    int rc = make_plan(pool, st, Hq, rows, rows_max, tree != nullptr, &plan, scale, win);
    if (rc != TF_OK)
        return rc;
    plan.p.wait_limit = faults.wait_limit;
    plan.p.withhold = faults.withhold;
    if (!std::isfinite(scale))
        return TF_EINVAL;
    if (st->n_streams == 0)
        return TF_OK;  // nothing is read or written: the buffers may be null
    if (!q || !out || !ws || !aligned16(q) || !aligned16(out) || !aligned16(ws))
        return TF_EINVAL;
    if (ws_bytes < plan.ws_bytes)
        return TF_ENOSPACE;
    AttnParams &p = plan.p;
    p.k_pool = static_cast<const __nv_bfloat16 *>(pool->k_pool);
    p.v_pool = static_cast<const __nv_bfloat16 *>(pool->v_pool);
    p.table = st->table;
    p.lens = st->lens;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.tree = tree;
    p.out = out;
    char *wsb = static_cast<char *>(ws);
    p.flags = reinterpret_cast<uint32_t *>(wsb);
    p.total_tiles = reinterpret_cast<long long *>(wsb + kWsTotalOffset);
    p.first_tile = reinterpret_cast<long long *>(wsb + kWsHeaderBytes);
    p.part = reinterpret_cast<float *>(wsb + ws_part_offset(p.S));
    p.scale_log2 = scale * 1.4426950408889634f;  // log2(e)
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (plan.kernel == Kernel::kWin) {
        e = launch_attn_win(plan.p, plan.grid, s);
    } else if (win) {
        e = launch_tensor_core(plan.p, plan, s);
    } else if (plan.kernel != Kernel::kSimt) {
        e = launch_tensor_core(p, plan, s);
    } else if (p.D == 128) {
        e = launch_attn_simt<128>(p, plan.grid, s);
        if (e == cudaSuccess)
            e = launch_attn_merge<128>(p, s);
    } else {
        e = launch_attn_simt<512>(p, plan.grid, s);
        if (e == cudaSuccess)
            e = launch_attn_merge<512>(p, s);
    }
    return e == cudaSuccess ? TF_OK : TF_ECUDA;
}

// Pages and entries of a table row at most: the kernels step past the last
// one by up to a block's 4,096, in 32 bits.
constexpr int32_t kMaxPages = INT32_MAX - 8192;

// The checks every page call shares; fills the common parameters.
int check_pages(const tf_kv_pages *pages, int32_t *table, int32_t stride, int32_t n_streams,
                uint32_t *status, PagesParams *p)
{
    if (!pages || pages->n_pages < 1 || pages->n_pages > kMaxPages || pages->page_size < 1 ||
        !pages->refs || !aligned16(pages->refs) || !aligned4(status))
        return TF_EINVAL;
    if (n_streams < 0 || stride < 1 || stride > kMaxPages || (int64_t)n_streams * stride > INT32_MAX)
        return TF_EINVAL;
    if (n_streams > 0 && (!table || !aligned4(table)))
        return TF_EINVAL;
    *p = PagesParams{};
    p->refs = pages->refs;
    p->n_pages = pages->n_pages;
    p->P = pages->page_size;
    p->table = table;
    p->stride = stride;
    p->S = n_streams;
    p->status = status;
    return TF_OK;
}

// Entries a list of `bytes` bytes can hold beside its head.
int64_t move_cap(size_t bytes)
{
    const size_t n = bytes / TF_MOVE_BYTES;
    return n == 0 ? -1 : n - 1 > INT32_MAX / 4 ? INT32_MAX / 4 : (int64_t)n - 1;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? TF_OK : TF_ECUDA; }

}  // namespace
}  // namespace tfp

using namespace tfp;

extern "C" {

int tf_kv_put_rows(const tf_kv_pool *pool, const tf_streams *streams, const void *k_rows,
                   const void *v_rows, int32_t rows, void *stream)
{
    int rc = check_pool_streams(pool, streams);
    if (rc != TF_OK)
        return rc;
    if (rows < 1 || streams->max_len < rows)
        return TF_EINVAL;
    if (streams->n_streams == 0)
        return TF_OK;
    if (!k_rows || !v_rows || !aligned16(k_rows) || !aligned16(v_rows))
        return TF_EINVAL;
    PutParams p;
    p.k_pool = static_cast<__nv_bfloat16 *>(pool->k_pool);
    p.v_pool = static_cast<__nv_bfloat16 *>(pool->v_pool);
    p.table = streams->table;
    p.lens = streams->lens;
    p.k_rows = static_cast<const __nv_bfloat16 *>(k_rows);
    p.v_rows = static_cast<const __nv_bfloat16 *>(v_rows);
    p.n_pages = pool->n_pages;
    p.Hkv = pool->n_kv_heads;
    p.P = pool->page_size;
    p.D = pool->head_dim;
    p.table_stride = streams->table_stride;
    p.S = streams->n_streams;
    p.W = rows;
    return launch_kv_put(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? TF_OK : TF_ECUDA;
}

int tf_kv_put_rows_rope(const tf_kv_pool *pool, const tf_streams *streams, const tf_rope *rope,
                        const int32_t *positions, const void *q, int64_t q_stride, void *q_out,
                        int32_t n_q_heads, const void *k_rows, int64_t k_stride,
                        const void *v_rows, int64_t v_stride, int32_t rows, void *stream)
{
    int rc = check_pool_streams(pool, streams);
    if (rc != TF_OK)
        return rc;
    if (rows < 1 || streams->max_len < rows || n_q_heads < 0 || n_q_heads > (1 << 16) || !rope)
        return TF_EINVAL;
    if (rope->rotary_dim < 2 || rope->rotary_dim > pool->head_dim || rope->rotary_dim % 2 != 0 ||
        rope->n_axes < 1 || rope->n_axes > 4 || (rope->adjacent != 0 && rope->adjacent != 1))
        return TF_EINVAL;
    RopeParams p;
    for (int i = 0; i < 256; ++i)
        p.pair_axis[i] = 0;
    for (int i = 0; rope->pair_axis && i < rope->rotary_dim / 2; ++i) {
        if (rope->pair_axis[i] >= rope->n_axes)
            return TF_EINVAL;
        p.pair_axis[i] = rope->pair_axis[i];
    }
    if (((int64_t)n_q_heads + 2 * (int64_t)pool->n_kv_heads) * pool->head_dim > INT32_MAX)
        return TF_EINVAL;
    const int64_t q_row = (int64_t)n_q_heads * pool->head_dim;
    const int64_t kv_row = (int64_t)pool->n_kv_heads * pool->head_dim;
    if ((n_q_heads > 0 && (q_stride < q_row || q_stride % 8 != 0)) || k_stride < kv_row ||
        k_stride % 8 != 0 || v_stride < kv_row || v_stride % 8 != 0)
        return TF_EINVAL;
    if (n_q_heads > 0 && q == q_out && q != nullptr && q_stride != q_row)
        return TF_EINVAL;
    if (streams->n_streams == 0)
        return TF_OK;
    if (!rope->inv_freq || !aligned4(rope->inv_freq) || !positions || !aligned4(positions) || !k_rows ||
        !v_rows || !aligned16(k_rows) || !aligned16(v_rows))
        return TF_EINVAL;
    if (n_q_heads > 0 && (!q || !q_out || !aligned16(q) || !aligned16(q_out)))
        return TF_EINVAL;
    p.k_pool = static_cast<__nv_bfloat16 *>(pool->k_pool);
    p.v_pool = static_cast<__nv_bfloat16 *>(pool->v_pool);
    p.table = streams->table;
    p.lens = streams->lens;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k_rows);
    p.v = static_cast<const __nv_bfloat16 *>(v_rows);
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.positions = positions;
    p.inv_freq = rope->inv_freq;
    p.q_stride = n_q_heads > 0 ? q_stride : 0;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.n_pages = pool->n_pages;
    p.Hkv = pool->n_kv_heads;
    p.Hq = n_q_heads;
    p.P = pool->page_size;
    p.D = pool->head_dim;
    p.table_stride = streams->table_stride;
    p.S = streams->n_streams;
    p.W = rows;
    p.max_len = streams->max_len;
    p.rotary = rope->rotary_dim;
    p.n_axes = rope->n_axes;
    p.adjacent = rope->adjacent;
    return launch_kv_rope(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? TF_OK : TF_ECUDA;
}

int tf_kv_copy_state(const tf_kv_pool *src_pool, const tf_streams *src,
                     const tf_kv_pool *dst_pool, const int32_t *dst_table,
                     int32_t dst_table_stride, uint32_t *status, void *stream)
{
    int rc = check_pool_streams(src_pool, src);
    if (rc != TF_OK)
        return rc;
    if (!dst_pool || dst_pool->n_pages < 1 || dst_pool->page_size < 1)
        return TF_EINVAL;
    if (dst_pool->n_kv_heads != src_pool->n_kv_heads || dst_pool->head_dim != src_pool->head_dim)
        return TF_EINVAL;
    if (!dst_pool->k_pool || !dst_pool->v_pool || !aligned16(dst_pool->k_pool) ||
        !aligned16(dst_pool->v_pool))
        return TF_EINVAL;
    if (dst_table_stride < 1 ||
        (int64_t)src->max_len > (int64_t)dst_table_stride * dst_pool->page_size ||
        (int64_t)src->n_streams * dst_table_stride > INT32_MAX)
        return TF_EINVAL;
    if (src->n_streams > 0 && (!dst_table || !aligned4(dst_table)))
        return TF_EINVAL;
    if (!aligned4(status))
        return TF_EINVAL;
    if (src->n_streams == 0)
        return TF_OK;
    CopyParams p;
    p.src_k = static_cast<const __nv_bfloat16 *>(src_pool->k_pool);
    p.src_v = static_cast<const __nv_bfloat16 *>(src_pool->v_pool);
    p.dst_k = static_cast<__nv_bfloat16 *>(dst_pool->k_pool);
    p.dst_v = static_cast<__nv_bfloat16 *>(dst_pool->v_pool);
    p.src_table = src->table;
    p.dst_table = dst_table;
    p.lens = src->lens;
    p.status = status;
    p.src_stride = src->table_stride;
    p.dst_stride = dst_table_stride;
    p.src_P = src_pool->page_size;
    p.dst_P = dst_pool->page_size;
    p.src_n_pages = src_pool->n_pages;
    p.dst_n_pages = dst_pool->n_pages;
    p.Hkv = src_pool->n_kv_heads;
    p.D = src_pool->head_dim;
    p.S = src->n_streams;
    p.max_len = src->max_len;
    p.chunk = copy_chunk_positions(p.D);
    p.n_chunks = (src->max_len + p.chunk - 1) / p.chunk;
    return launch_kv_copy(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? TF_OK : TF_ECUDA;
}

int tf_kv_pages_fork(const tf_kv_pages *pages, const int32_t *src_table, int32_t src_stride,
                     const int32_t *src_lens, int32_t n_src, const int32_t *parents, int32_t n_dst,
                     int32_t *dst_table, int32_t dst_stride, int32_t *dst_lens, uint32_t *status,
                     void *stream)
{
    PagesParams p;
    const int rc =
        check_pages(pages, const_cast<int32_t *>(src_table), src_stride, n_src, status, &p);
    if (rc != TF_OK)
        return rc;
    if (n_dst < 0 || dst_stride < 1 || dst_stride > kMaxPages ||
        (int64_t)n_dst * dst_stride > INT32_MAX)
        return TF_EINVAL;
    if (n_src > 0 && (!src_lens || !aligned4(src_lens)))
        return TF_EINVAL;
    if (n_dst == 0)
        return TF_OK;
    if (!parents || !dst_table || !dst_lens || !aligned4(parents) || !aligned4(dst_table) ||
        !aligned4(dst_lens))
        return TF_EINVAL;
    p.lens = src_lens;
    p.parents = parents;
    p.dst_table = dst_table;
    p.dst_lens = dst_lens;
    p.dst_stride = dst_stride;
    return status_of(launch_pages_fork(p, n_dst, static_cast<cudaStream_t>(stream)));
}

int tf_kv_pages_free(const tf_kv_pages *pages, int32_t *table, int32_t table_stride,
                     int32_t n_streams, const int32_t *first, const int32_t *end, uint32_t *status,
                     void *stream)
{
    PagesParams p;
    const int rc = check_pages(pages, table, table_stride, n_streams, status, &p);
    if (rc != TF_OK || n_streams == 0)
        return rc;
    if (!aligned4(first) || !aligned4(end))
        return TF_EINVAL;
    p.first = first;
    p.end = end;
    return status_of(launch_pages_free(p, false, static_cast<cudaStream_t>(stream)));
}

int tf_kv_pages_free_window(const tf_kv_pages *pages, int32_t *table, int32_t table_stride,
                            const int32_t *lens, int32_t n_streams, int32_t window, int32_t sinks,
                            uint32_t *status, void *stream)
{
    PagesParams p;
    const int rc = check_pages(pages, table, table_stride, n_streams, status, &p);
    if (rc != TF_OK)
        return rc;
    if (window < 1 || sinks < 0 || (n_streams > 0 && (!lens || !aligned4(lens))))
        return TF_EINVAL;
    if (n_streams == 0)
        return TF_OK;
    p.lens = lens;
    p.window = window;
    p.sinks = sinks;
    return status_of(launch_pages_free(p, true, static_cast<cudaStream_t>(stream)));
}

int tf_kv_pages_grow(const tf_kv_pages *pages, int32_t *table, int32_t table_stride,
                     const int32_t *lens, int32_t n_streams, int32_t rows, void *moves,
                     size_t moves_bytes, uint32_t *status, void *stream)
{
    PagesParams p;
    const int rc = check_pages(pages, table, table_stride, n_streams, status, &p);
    if (rc != TF_OK)
        return rc;
    if (rows < 1 || (n_streams > 0 && (!lens || !aligned4(lens))) || !moves || !aligned16(moves))
        return TF_EINVAL;
    const int64_t per_stream = ((int64_t)rows + p.P - 2) / p.P + 1;
    const int64_t cap = move_cap(moves_bytes);
    if (cap < 0 || per_stream * n_streams > cap)
        return TF_ENOSPACE;
    p.lens = lens;
    p.rows = rows;
    p.per_stream = static_cast<int32_t>(per_stream);
    p.moves = static_cast<int4 *>(moves);
    return status_of(launch_pages_grow(p, static_cast<cudaStream_t>(stream)));
}

int tf_kv_pages_compact(const tf_kv_pages *pages, int32_t *table, int32_t table_stride,
                        int32_t n_streams, void *moves, size_t moves_bytes, uint32_t *status,
                        void *stream)
{
    PagesParams p;
    const int rc = check_pages(pages, table, table_stride, n_streams, status, &p);
    if (rc != TF_OK)
        return rc;
    if (!moves || !aligned16(moves))
        return TF_EINVAL;
    if (move_cap(moves_bytes) < p.n_pages / 2)
        return TF_ENOSPACE;
    p.moves = static_cast<int4 *>(moves);
    return status_of(launch_pages_compact(p, static_cast<cudaStream_t>(stream)));
}

int tf_kv_pages_move(const tf_kv_pool *pool, const void *moves, size_t moves_bytes,
                     uint32_t *status, void *stream)
{
    // (the pool's checks are those of a call without streams)
    const tf_streams none{nullptr, 1, nullptr, 0, 1};
    int rc = check_pool_streams(pool, &none);
    if (rc != TF_OK)
        return rc;
    const int64_t cap = move_cap(moves_bytes);
    if (!moves || !aligned16(moves) || cap < 0 || !aligned4(status))
        return TF_EINVAL;
    int sms = 0;
    rc = device_sm_count(&sms);
    if (rc != TF_OK)
        return rc;
    MoveParams p{};
    p.k_pool = pool->k_pool;
    p.v_pool = pool->v_pool;
    p.moves = static_cast<const int32_t *>(moves);
    p.status = status;
    p.n_pages = pool->n_pages;
    p.Hkv = pool->n_kv_heads;
    p.P = pool->page_size;
    p.D = pool->head_dim;
    p.cap = static_cast<int32_t>(cap);
    return status_of(launch_pages_move(p, sms, static_cast<cudaStream_t>(stream)));
}

size_t tf_paged_attn_workspace_bytes(const tf_kv_pool *pool, const tf_streams *streams,
                                     int32_t n_q_heads, int32_t rows)
{
    Plan plan;
    if (make_plan(pool, streams, n_q_heads, rows, 4096, false, &plan) != TF_OK)
        return 0;
    return plan.ws_any;
}

int tf_paged_attn_decode(const tf_kv_pool *pool, const tf_streams *streams, const void *q,
                         int32_t n_q_heads, float scale, float *out, void *workspace,
                         size_t workspace_bytes, void *stream)
{
    return attn_call(pool, streams, q, n_q_heads, 1, 1, nullptr, scale, out, workspace,
                     workspace_bytes, stream);
}

int tf_paged_attn_verify(const tf_kv_pool *pool, const tf_streams *streams, const void *q,
                         int32_t n_q_heads, int32_t rows, float scale, float *out,
                         void *workspace, size_t workspace_bytes, void *stream)
{
    return attn_call(pool, streams, q, n_q_heads, rows, 8, nullptr, scale, out, workspace,
                     workspace_bytes, stream);
}

int tf_paged_attn_verify_tree(const tf_kv_pool *pool, const tf_streams *streams, const void *q,
                              int32_t n_q_heads, int32_t rows, const uint8_t *tree_masks,
                              float scale, float *out, void *workspace, size_t workspace_bytes,
                              void *stream)
{
    if (streams && streams->n_streams > 0 && !tree_masks)
        return TF_EINVAL;
    return attn_call(pool, streams, q, n_q_heads, rows, 8, tree_masks, scale, out, workspace,
                     workspace_bytes, stream);
}

int tf_paged_attn_prompt(const tf_kv_pool *pool, const tf_streams *streams, const void *q,
                         int32_t n_q_heads, int32_t rows, float scale, float *out,
                         void *workspace, size_t workspace_bytes, void *stream)
{
    return attn_call(pool, streams, q, n_q_heads, rows, 4096, nullptr, scale, out, workspace,
                     workspace_bytes, stream);
}

size_t tf_paged_attn_window_workspace_bytes(const tf_kv_pool *pool, const tf_streams *streams,
                                            int32_t n_q_heads, int32_t rows, int32_t window,
                                            int32_t sinks)
{
    const Window win{window, sinks, 0};
    Plan plan;
    if (make_plan(pool, streams, n_q_heads, rows, 4096, false, &plan, 1.f, &win) != TF_OK)
        return 0;
    return plan.ws_any;
}

int tf_paged_attn_decode_window(const tf_kv_pool *pool, const tf_streams *streams, const void *q,
                                int32_t n_q_heads, int32_t window, int32_t sinks, float scale,
                                float *out, void *workspace, size_t workspace_bytes, void *stream)
{
    const Window win{window, sinks, 0};
    return attn_call(pool, streams, q, n_q_heads, 1, 1, nullptr, scale, out, workspace,
                     workspace_bytes, stream, Faults{}, &win);
}

int tf_paged_attn_verify_window(const tf_kv_pool *pool, const tf_streams *streams, const void *q,
                                int32_t n_q_heads, int32_t rows, int32_t window, int32_t sinks,
                                float scale, float *out, void *workspace, size_t workspace_bytes,
                                void *stream)
{
    const Window win{window, sinks, 0};
    return attn_call(pool, streams, q, n_q_heads, rows, 8, nullptr, scale, out, workspace,
                     workspace_bytes, stream, Faults{}, &win);
}

int tf_paged_attn_prompt_window(const tf_kv_pool *pool, const tf_streams *streams, const void *q,
                                int32_t n_q_heads, int32_t rows, int32_t window, int32_t sinks,
                                float scale, float *out, void *workspace, size_t workspace_bytes,
                                void *stream)
{
    const Window win{window, sinks, 0};
    return attn_call(pool, streams, q, n_q_heads, rows, 4096, nullptr, scale, out, workspace,
                     workspace_bytes, stream, Faults{}, &win);
}

int tf_testing_paged_attn(const tf_kv_pool *pool, const tf_streams *streams, const void *q,
                          int32_t n_q_heads, int32_t rows, float scale, float *out,
                          void *workspace, size_t workspace_bytes, int64_t wait_limit_cycles,
                          int32_t withhold, void *stream)
{
    if (wait_limit_cycles < 1000000 || wait_limit_cycles > kWaitLimitCycles)
        return TF_EINVAL;
    if (withhold != 0 && withhold != 1)
        return TF_EINVAL;
    Faults f;
    f.wait_limit = wait_limit_cycles;
    f.withhold = withhold;
    return attn_call(pool, streams, q, n_q_heads, rows, 4096, nullptr, scale, out, workspace,
                     workspace_bytes, stream, f);
}

int tf_testing_paged_attn_window(const tf_kv_pool *pool, const tf_streams *streams, const void *q,
                                 int32_t n_q_heads, int32_t rows, int32_t window, int32_t sinks,
                                 float scale, float *out, void *workspace, size_t workspace_bytes,
                                 int32_t kernel, int64_t wait_limit_cycles, int32_t withhold,
                                 void *stream)
{
    if (wait_limit_cycles < 1000000 || wait_limit_cycles > kWaitLimitCycles)
        return TF_EINVAL;
    if ((withhold != 0 && withhold != 1) || kernel < 0 || kernel > 2)
        return TF_EINVAL;
    Faults f;
    f.wait_limit = wait_limit_cycles;
    f.withhold = withhold;
    const Window win{window, sinks, kernel};
    return attn_call(pool, streams, q, n_q_heads, rows, 4096, nullptr, scale, out, workspace,
                     workspace_bytes, stream, f, &win);
}

int tf_workspace_status(void *workspace, uint32_t *flags, void *stream)
{
    if (!workspace || !flags)
        return TF_EINVAL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint32_t host = 0;
    if (cudaMemcpyAsync(&host, workspace, sizeof host, cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return TF_ECUDA;
    if (cudaMemsetAsync(workspace, 0, sizeof host, s) != cudaSuccess)
        return TF_ECUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess)
        return TF_ECUDA;
    *flags = host;
    return TF_OK;
}

const char *tf_status_str(int status)
{
    switch (status) {
    case TF_OK:
        return "TF_OK";
    case TF_EINVAL:
        return "TF_EINVAL: invalid argument";
    case TF_EUNSUPPORTED:
        return "TF_EUNSUPPORTED: shape not supported by this library";
    case TF_ENOSPACE:
        return "TF_ENOSPACE: workspace too small";
    case TF_ECUDA:
        return "TF_ECUDA: CUDA launch or query failed";
    default:
        return "unknown status";
    }
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Decode without a caller-provided workspace.
//
// Some callers cannot allocate device memory for a workspace: a plug-in
// hosted by an inference engine that hands it only its input and output
// buffers and owns every allocation itself, or a serving loop that must not
// call cudaMalloc once it is running (cudaMalloc can synchronise the device
// and can fail under memory pressure).  For them the split-context scratch
// lives in one file-scope device array of kStaticScratchBytes, which every
// GPU that loads this library keeps until the process exits.
namespace tfp {
namespace {

constexpr size_t kStaticScratchBytes = size_t(8) << 20;  // 8 MiB per device

static __device__ __align__(256) unsigned char g_decode_scratch[kStaticScratchBytes];

// Device address of g_decode_scratch on the current device.  In host code
// the array's name is only a host-side stand-in, so its device address is
// looked up once per device (with that device current) and cached.
int static_scratch_address(void **out)
{
    static std::mutex mu;
    static void *addr[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return TF_ECUDA;
    std::lock_guard<std::mutex> lock(mu);
    if (addr[dev] == nullptr) {
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_decode_scratch) != cudaSuccess || p == nullptr)
            return TF_ECUDA;
        addr[dev] = p;
    }
    *out = addr[dev];
    return TF_OK;
}

}  // namespace
}  // namespace tfp

extern "C" int tf_paged_attn_decode_noalloc(const tf_kv_pool *pool, const tf_streams *streams,
                                            const void *q, int32_t n_q_heads, float scale,
                                            float *out, void *stream)
{
    using namespace tfp;
    Plan plan;
    int rc = make_plan(pool, streams, n_q_heads, 1, 1, false, &plan, scale);
    if (rc != TF_OK)
        return rc;
    if (!std::isfinite(scale))
        return TF_EINVAL;
    // as tf_paged_attn_decode: a call with no streams reads and writes
    // nothing, and its buffers may be null
    if (streams->n_streams == 0)
        return TF_OK;
    if (!q || !out || !aligned16(q) || !aligned16(out))
        return TF_EINVAL;
    if (plan.ws_bytes > kStaticScratchBytes)
        return TF_ENOSPACE;
    void *ws = nullptr;
    rc = static_scratch_address(&ws);
    if (rc != TF_OK)
        return rc;
    // Nothing in the scratch needs clearing: the kernels write every partial
    // and the header's tile counts before reading them.  The header's status
    // and wait-site words only collect bits (ORed in by the kernels) that no
    // kernel reads and this call does not report, so they are left as they
    // are; their contents are unspecified.
    return attn_call(pool, streams, q, n_q_heads, 1, 1, nullptr, scale, out, ws, kStaticScratchBytes,
                     stream);
}
