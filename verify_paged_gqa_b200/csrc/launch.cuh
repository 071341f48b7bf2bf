// launch.cuh -- host-side launchers of the kernels (one per translation unit).
#pragma once

#include "common.cuh"

#include <atomic>

namespace tfp {

// Raises `kernel`'s dynamic shared memory limit to `bytes`, once per device
// (done[dev] records it).  Host threads making their first launches at once
// may each set the same attribute, which is harmless; the flags are atomics,
// so that race is well defined.
template <class Kernel>
cudaError_t set_smem_limit_once(Kernel kernel, size_t bytes, std::atomic<bool> (&done)[kMaxDevices])
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_acquire))
        return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess)
        done[dev].store(true, std::memory_order_release);
    return e;
}

// Launches `kernel` as a programmatic dependent of the previous kernel in the
// stream: its blocks may be scheduled while that kernel finishes, and wait
// for it in the kernel (wait_prior_grid) before reading its outputs.
template <class Kernel, class Arg>
cudaError_t launch_dependent(Kernel kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                             const Arg &arg)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, arg);
}

struct PutParams {
    __nv_bfloat16 *k_pool;
    __nv_bfloat16 *v_pool;
    const int32_t *table;
    const int32_t *lens;
    const __nv_bfloat16 *k_rows;
    const __nv_bfloat16 *v_rows;
    int32_t n_pages, Hkv, P, D;
    int32_t table_stride, S, W;
};

cudaError_t launch_kv_put(const PutParams &p, cudaStream_t stream);

// The row write with rotary positions (kv_rope.cu).
struct RopeParams {
    __nv_bfloat16 *k_pool;
    __nv_bfloat16 *v_pool;
    const int32_t *table;
    const int32_t *lens;
    const __nv_bfloat16 *q;       // rows of Hq heads, q_stride elements apart
    const __nv_bfloat16 *k;
    const __nv_bfloat16 *v;
    __nv_bfloat16 *q_out;         // [S][W][Hq][D]
    const int32_t *positions;     // [S][W][n_axes]
    const float *inv_freq;        // [rotary / 2]
    int64_t q_stride, k_stride, v_stride;
    int32_t n_pages, Hkv, Hq, P, D;
    int32_t table_stride, S, W, max_len;
    int32_t rotary, n_axes, adjacent;
    uint8_t pair_axis[256];       // axis of pair i
};

cudaError_t launch_kv_rope(const RopeParams &p, cudaStream_t stream);

// The state copy (kv_copy.cu): positions [0, lens[s]) of every KV head from
// the source pool's pages to the destination pool's pages.
struct CopyParams {
    const __nv_bfloat16 *src_k;
    const __nv_bfloat16 *src_v;
    __nv_bfloat16 *dst_k;
    __nv_bfloat16 *dst_v;
    const int32_t *src_table;
    const int32_t *dst_table;
    const int32_t *lens;
    uint32_t *status;              // TF_DEV_* bits are ORed in (may be null)
    int32_t src_stride, dst_stride, src_P, dst_P, src_n_pages, dst_n_pages;
    int32_t Hkv, D, S, max_len;
    int32_t chunk;                 // positions per block
    int32_t n_chunks;              // blocks per (stream, KV head): ceil(max_len / chunk)
};

int copy_chunk_positions(int head_dim);
cudaError_t launch_kv_copy(const CopyParams &p, cudaStream_t stream);

// The pages' bookkeeping (kv_pages.cu); each call uses what it needs.
struct PagesParams {
    int32_t *refs;              // table entries that hold each page; 16-byte aligned
    int32_t n_pages, P;
    int32_t *table;             // [S][stride], -1: no page
    const int32_t *lens;
    int32_t stride, S;
    uint32_t *status;           // TF_DEV_* bits are ORed in (may be null)
    // fork
    const int32_t *parents;
    int32_t *dst_table, *dst_lens;
    int32_t dst_stride;
    // free
    const int32_t *first, *end;  // may be null: from the first, to the last entry
    int32_t window, sinks;
    // grow and compact: the list of page moves, entry 0 its head
    int4 *moves;
    int32_t rows, per_stream;    // grow: new positions, and the pages they can touch
};

cudaError_t launch_pages_fork(const PagesParams &p, int n_dst, cudaStream_t stream);
cudaError_t launch_pages_free(const PagesParams &p, bool window, cudaStream_t stream);
cudaError_t launch_pages_grow(const PagesParams &p, cudaStream_t stream);
cudaError_t launch_pages_compact(const PagesParams &p, cudaStream_t stream);

struct MoveParams {
    void *k_pool;
    void *v_pool;
    const int32_t *moves;
    uint32_t *status;
    int32_t n_pages, Hkv, P, D;
    int32_t cap;                 // entries the list can hold
    int32_t pieces, per_head;    // (set by the launcher) runs per page and KV head
};

cudaError_t launch_pages_move(MoveParams p, int sms, cudaStream_t stream);

// Rows per row block of the CUDA-core partial kernel.
constexpr int kSimtRows = 4;

// Sliding-window kernel of row blocks of 4, 8 or 16 rows (attn_win.cu): grid =
// units * p.whole blocks in clusters of p.whole = win_split's C, one per unit.
constexpr int kMaxCluster = 8;
struct WinSplit {
    int C;
    int64_t cost;  // in chunks of 16 positions, one after another
};
WinSplit win_split(const WinParams &p, int64_t units);
cudaError_t launch_attn_win(const WinParams &p, int grid, cudaStream_t stream);

template <int D>
size_t simt_smem_bytes();
template <int D>
cudaError_t launch_attn_simt(const AttnParams &p, int grid, cudaStream_t stream);
template <int D, class P>
cudaError_t launch_attn_merge(const P &p, cudaStream_t stream);  // D 128, 256, 512

// Prompt tensor-core partial kernel (tcgen05): row blocks of prompt_rows()
// rows on the QK MMA's M, PV transposed.
int prompt_rows();
bool prompt_supported(const AttnParams &p);
cudaError_t launch_attn_prompt(const AttnParams &p, int grid, cudaStream_t stream);
cudaError_t launch_attn_prompt(const WinParams &p, int grid, cudaStream_t stream);

// Position-major tensor-core partial kernel: key positions on the MMA's M,
// row blocks of pm_rows() rows (0: not supported for these arguments), kPmWideRows
// at head dims 256 and 512.  More than 64 rows per KV head at head dim 128 are
// the prompt kernel's, unless `any_count`.
constexpr int kPmWideRows = 32;
int pm_rows(const AttnParams &p, bool any_count);
cudaError_t launch_attn_pm(const AttnParams &p, int grid, cudaStream_t stream);
cudaError_t launch_attn_pm(const WinParams &p, int grid, cudaStream_t stream);

}  // namespace tfp
