// libpa, one-query window attention: C ABI of pa_decode_window and
// pa_decode_q8 and their workspace.  Host code here only validates arguments,
// sizes the grid and launches; the arithmetic runs in
// window_decode_kernel.cuh.  Nothing here allocates device memory.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/pa_window.h"
#include "host_common.cuh"
#include "window_decode_kernel.cuh"
#include "window_host.cuh"
#include "window_maps.cuh"

namespace {

// Partial results (two per range: its first and its last unit, the only ones
// that can straddle ranges), then one merge counter per unit.  The slots have
// room for the most any call needs, so that the counters of calls that
// share a workspace always lie in the same place.
struct WindowWorkspace {
    size_t ml_off, ticket_off, total;
};

// Query heads of a unit: 4 for groups of up to 4, else 8, or 16 for groups of
// more than 8 when that leaves units enough (measured in
// window_decode_kernel.cuh).
int unit_heads(int num_seqs, int num_kv_heads, int group)
{
    constexpr int64_t kFewUnits = 32;
    if (group <= 4)
        return 4;
    return group <= 8 || int64_t(num_seqs) * num_kv_heads * ((group + 15) / 16) <= kFewUnits ? 8 : 16;
}

WindowWorkspace window_workspace(int num_seqs, int num_heads, int num_kv_heads)
{
    WindowWorkspace w{};
    const int group = num_heads / num_kv_heads;
    const size_t slots = size_t(pa::kWdSlots);
    const size_t units = size_t(num_seqs) * num_kv_heads * ((group + 7) / 8);
    w.ml_off = align256(slots * 16 * 128 * sizeof(float));
    w.ticket_off = w.ml_off + align256(slots * 16 * sizeof(float2));
    w.total = w.ticket_off + align256((units > 0 ? units : 1) * sizeof(unsigned));
    return w;
}

template <pa::KvStore kStore, int D, int kHeads>
pa_status launch_window(const pa::WindowDecodeParams &p, const void *k, const void *v,
                        cudaStream_t stream)
{
    using W = pa::WindowTraits<kStore, D>;
    constexpr auto kernel = pa::window_decode_kernel<kStore, D, kHeads>;
    static std::atomic<int> grid_for[kMaxDevices];  // 0 = not configured yet
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return PA_ERR_CUDA;
    int grid = grid_for[dev].load(std::memory_order_acquire);
    if (grid == 0) {
        int sms = 0, per_sm = 0;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 W::kSmem) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, pa::kWdThreads,
                                                          W::kSmem) != cudaSuccess)
            return PA_ERR_CUDA;
        grid = std::min(sms * std::max(per_sm, 1), pa::kWdMaxCtas);
        grid_for[dev].store(grid, std::memory_order_release);
    }
    CUtensorMap tm_k, tm_v;
    const uint64_t rows = (uint64_t(p.num_blocks) * p.kv_heads) << p.log2_bs;
    const uint32_t box = uint32_t(std::min(1 << p.log2_bs, W::kTile));
    const bool ok = [&] {
        if constexpr (W::kEight)
            return line_map(&tm_k, k, rows * D / 128, box * D / 128) &&
                   line_map(&tm_v, v, rows * D / 128, box * D / 128);
        else
            return cache_map<D>(&tm_k, k, rows, box) && cache_map<D>(&tm_v, v, rows, box);
    }();
    return ok && launch_pdl(kernel, dim3(unsigned(grid)), dim3(pa::kWdThreads), W::kSmem, stream, tm_k,
                            tm_v, p) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

pa_status window_decode(void *out, const void *q, const void *k, const void *v,
                        const float *scales, bool eight, const int32_t *block_tables,
                        int max_blocks_per_seq, const int32_t *context_lens, int max_context_len,
                        int window, int num_sinks, int num_seqs, int num_heads, int num_kv_heads,
                        int head_dim, int block_size, int num_blocks, int dtype, int kv_type,
                        float scale, void *workspace, size_t workspace_bytes, pa_stream_t stream)
{
    if (num_seqs < 0 || num_blocks <= 0 || max_context_len < 0 || max_blocks_per_seq < 0 ||
        window < 1 || num_sinks < 0 || !valid_dtype(dtype) || (eight && !valid_kv8(kv_type)) ||
        !valid_heads(num_heads, num_kv_heads) || !std::isfinite(scale))
        return PA_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || !supported_block_size(block_size))
        return PA_ERR_UNSUPPORTED;
    if (int64_t(max_context_len) > int64_t(max_blocks_per_seq) * block_size || num_seqs > 65535 ||
        max_context_len > (1 << 30))
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0)
        return PA_OK;
    if (!out || !q || !k || !v || !context_lens || !block_tables || (eight && !scales))
        return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(scales) ||
        (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
        (reinterpret_cast<uintptr_t>(context_lens) & 3u))
        return PA_ERR_INVALID_ARG;
    const WindowWorkspace w = window_workspace(num_seqs, num_heads, num_kv_heads);
    if (!workspace || workspace_bytes < w.total)
        return PA_ERR_WORKSPACE;
    if (!aligned16(workspace))
        return PA_ERR_INVALID_ARG;

    // the tensor maps address the caches in groups of 8 rows or lines of 128
    // bytes; the work is counted in 64 bits
    const int64_t cache_bytes = int64_t(num_blocks) * num_kv_heads * block_size * head_dim *
                                (eight ? 1 : 2);
    if (cache_bytes / (eight ? 128 : 16 * head_dim) > INT32_MAX ||
        int64_t(num_seqs) * num_heads * (max_context_len / 16 + 1) > (int64_t(1) << 50))
        return PA_ERR_INVALID_ARG;

    pa::WindowDecodeParams p{};
    p.out = out;
    p.q = q;
    p.scales = reinterpret_cast<const float2 *>(scales);
    p.tables = block_tables;
    p.lens = context_lens;
    p.max_blocks = max_blocks_per_seq;
    p.max_len = max_context_len;
    p.window = window;
    p.sinks = num_sinks;
    p.num_seqs = num_seqs;
    p.heads = num_heads;
    p.kv_heads = num_kv_heads;
    p.group = num_heads / num_kv_heads;
    const int per = unit_heads(num_seqs, num_kv_heads, p.group);
    p.row_tiles = (p.group + per - 1) / per;
    p.log2_bs = __builtin_ctz(unsigned(block_size));
    p.num_blocks = num_blocks;
    p.scale_heads = scale_heads(num_kv_heads);
    p.bf16 = dtype == PA_BF16;
    p.scale_log2 = float(double(scale) * 1.4426950408889634);
    p.shift = weight_shift(!eight && dtype == PA_BF16, max_context_len, window, num_sinks);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    p.part_o = reinterpret_cast<float4 *>(ws);
    p.part_ml = reinterpret_cast<float4 *>(ws + w.ml_off);
    p.tickets = reinterpret_cast<unsigned *>(ws + w.ticket_off);
    p.err = device_error_word();
    if (!p.err)
        return PA_ERR_CUDA;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return with_bool(head_dim == 128, [&](auto d128) {
        auto of = [&](auto heads) {
            constexpr int D = d128 ? 128 : 64, kHeads = heads;
            if (eight)
                return kv_type == PA_KV8_E4M3 ? launch_window<pa::KvStore::kE4m3, D, kHeads>(p, k, v, st)
                                              : launch_window<pa::KvStore::kInt8, D, kHeads>(p, k, v, st);
            return dtype == PA_BF16 ? launch_window<pa::KvStore::kBf16, D, kHeads>(p, k, v, st)
                                    : launch_window<pa::KvStore::kF16, D, kHeads>(p, k, v, st);
        };
        return per == 4    ? of(std::integral_constant<int, 4>{})
               : per == 8 ? of(std::integral_constant<int, 8>{})
                          : of(std::integral_constant<int, 16>{});
    });
}

} // namespace

extern "C" {

size_t pa_decode_window_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim)
{
    if (num_seqs < 0 || !valid_heads(num_heads, num_kv_heads) || head_dim <= 0)
        return window_workspace(1, 1, 1).total;
    return window_workspace(num_seqs, num_heads, num_kv_heads).total;
}

pa_status pa_decode_window(void *out, const void *q, const void *k_cache, const void *v_cache,
                           const int32_t *block_tables, int max_blocks_per_seq,
                           const int32_t *context_lens, int max_context_len, int window,
                           int num_sinks, int num_seqs, int num_heads, int num_kv_heads,
                           int head_dim, int block_size, int num_blocks, pa_dtype dtype,
                           float scale, void *workspace, size_t workspace_bytes,
                           pa_stream_t stream)
{
    return window_decode(out, q, k_cache, v_cache, nullptr, false, block_tables, max_blocks_per_seq,
                         context_lens, max_context_len, window, num_sinks, num_seqs, num_heads,
                         num_kv_heads, head_dim, block_size, num_blocks, dtype, 0, scale, workspace,
                         workspace_bytes, stream);
}

pa_status pa_decode_q8(void *out, const void *q, const void *k_codes, const void *v_codes,
                       const float *kv_scales, const int32_t *block_tables, int max_blocks_per_seq,
                       const int32_t *context_lens, int max_context_len, int window, int num_sinks,
                       int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                       int num_blocks, pa_dtype dtype, pa_kv8_type kv_type, float scale,
                       void *workspace, size_t workspace_bytes, pa_stream_t stream)
{
    return window_decode(out, q, k_codes, v_codes, kv_scales, true, block_tables,
                         max_blocks_per_seq, context_lens, max_context_len, window, num_sinks,
                         num_seqs, num_heads, num_kv_heads, head_dim, block_size, num_blocks, dtype,
                         kv_type, scale, workspace, workspace_bytes, stream);
}

} // extern "C"
