// libpa, multi-query window attention: C ABI of pa_prefill_window.  Host code
// here only validates arguments, encodes the TMA tensor maps and launches;
// the arithmetic runs in window_prefill_kernel.cuh.  Nothing here allocates
// device memory, and nothing is kept between calls.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/pa_window.h"
#include "host_common.cuh"
#include "window_host.cuh"
#include "window_maps.cuh"
#include "window_prefill_kernel.cuh"

namespace {

template <int D, bool kBf16>
pa_status launch_window_prefill(const pa::WindowPrefillParams &p, const void *q, const void *k_cache,
                                const void *v_cache, cudaStream_t stream)
{
    constexpr auto kernel = pa::window_prefill_kernel<D, kBf16>;
    constexpr int kSmem = int(pa::wp::Shape<D>::kSmem);
    static std::atomic<bool> configured[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
        return PA_ERR_CUDA;
    if (!configured[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
            cudaSuccess)
            return PA_ERR_CUDA;
        configured[dev].store(true, std::memory_order_release);
    }
    CUtensorMap tm_q, tm_k, tm_v;
    const uint64_t rows = (uint64_t(p.num_blocks) * p.kv_heads) << p.log2_bs;
    const uint32_t box = uint32_t(std::min(1 << p.log2_bs, pa::wp::kN));
    if (!swizzled_map<3>(&tm_q, q, {D, uint64_t(p.heads), uint64_t(p.num_rows)},
                         {D * 2, uint64_t(p.heads) * D * 2},
                         {64, uint32_t(p.group), uint32_t(p.tq)}) ||
        !cache_map<D>(&tm_k, k_cache, rows, box) || !cache_map<D>(&tm_v, v_cache, rows, box))
        return PA_ERR_CUDA;
    // at most one partly filled item a sequence and K/V head; CTAs without an
    // item end at once
    const int64_t per_item = int64_t(pa::wp::kTiles) * p.tq;
    const int64_t items =
        std::min(p.num_rows / per_item + p.num_seqs,
                 (int64_t(p.max_new) + per_item - 1) / per_item * p.num_seqs) *
        p.kv_heads;
    if (items > INT32_MAX)
        return PA_ERR_INVALID_ARG;
    return launch_pdl(kernel, dim3(unsigned(items)), dim3(pa::wp::kThreads), kSmem, stream, tm_q, tm_k,
                      tm_v, p) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

} // namespace

extern "C" pa_status pa_prefill_window(void *out, const void *q, const void *k_cache,
                                       const void *v_cache, const int32_t *block_tables,
                                       int max_blocks_per_seq, const int32_t *context_lens,
                                       int max_context_len, const int32_t *query_start_loc,
                                       int num_tokens, int max_query_len, int window, int num_sinks,
                                       int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                       int block_size, int num_blocks, pa_dtype dtype, float scale,
                                       pa_stream_t stream)
{
    if (num_seqs < 0 || num_tokens < 0 || max_query_len < 0 || num_blocks <= 0 || max_context_len < 0 ||
        max_blocks_per_seq < 0 || window < 1 || num_sinks < 0 || !valid_dtype(dtype) ||
        !valid_heads(num_heads, num_kv_heads))
        return PA_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || !supported_block_size(block_size))
        return PA_ERR_UNSUPPORTED;
    if (int64_t(max_context_len) > int64_t(max_blocks_per_seq) * block_size ||
        max_context_len > (1 << 30) || max_query_len > max_context_len || !std::isfinite(scale) ||
        !(scale > 0.f))
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_tokens == 0 || max_query_len == 0)
        return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start_loc)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
        (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
        (reinterpret_cast<uintptr_t>(context_lens) & 3u) ||
        (reinterpret_cast<uintptr_t>(query_start_loc) & 3u))
        return PA_ERR_INVALID_ARG;
    // the tensor maps address the caches in groups of 8 rows
    if (num_seqs > 65535 || int64_t(num_blocks) * num_kv_heads * (block_size / 8) > INT32_MAX)
        return PA_ERR_INVALID_ARG;

    pa::WindowPrefillParams p{};
    p.out = out;
    p.tables = block_tables;
    p.lens = context_lens;
    p.starts = query_start_loc;
    p.max_blocks = max_blocks_per_seq;
    p.max_len = max_context_len;
    p.max_new = max_query_len;
    p.window = window;
    p.sinks = num_sinks;
    p.num_seqs = num_seqs;
    p.heads = num_heads;
    p.kv_heads = num_kv_heads;
    p.group = num_heads / num_kv_heads;
    p.tq = pa::wp::kM / p.group;
    p.log2_bs = __builtin_ctz(unsigned(block_size));
    p.num_blocks = num_blocks;
    p.num_rows = num_tokens;
    p.scale_log2 = float(double(scale) * 1.4426950408889634);
    p.shift = weight_shift(dtype == PA_BF16, max_context_len, window, num_sinks);
    p.err = device_error_word();
    if (!p.err)
        return PA_ERR_CUDA;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return with_bool(head_dim == 128, [&](auto d128) {
        return with_bool(dtype == PA_BF16, [&](auto bf16) {
            return launch_window_prefill<d128 ? 128 : 64, bf16>(p, q, k_cache, v_cache, st);
        });
    });
}
