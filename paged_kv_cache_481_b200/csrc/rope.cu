// libpa, rotating cache writes: C ABI of pa_rope_and_cache and
// pa_rope_and_cache_q8.  Host code here only validates arguments and launches
// the kernels of rope_kernel.cuh.  Nothing here allocates device memory.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/pa_window.h"
#include "host_common.cuh"
#include "rope_kernel.cuh"
#include "window_host.cuh"

namespace {

// Arguments that the 16-bit and the 8-bit write share, checked and packed.
pa_status rope_params(pa::RopeParams &p, void *q_out, int64_t q_out_stride, const void *q,
                      int64_t q_stride, const void *key, int64_t key_stride, const void *value,
                      int64_t value_stride, void *k_cache, void *v_cache, const float *cos_sin,
                      int rotary_dim, int max_position, const int64_t *positions,
                      const int64_t *slot_mapping, int num_tokens, int num_heads, int num_kv_heads,
                      int head_dim, int block_size, int num_blocks, pa_dtype dtype)
{
    if (num_tokens < 0 || num_blocks <= 0 || max_position < 0 || !valid_dtype(dtype) ||
        !valid_heads(num_heads, num_kv_heads))
        return PA_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || !supported_block_size(block_size) || rotary_dim < 0 ||
        rotary_dim > head_dim || rotary_dim % 16 != 0)
        return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0)
        return PA_OK;
    const int64_t q_row = int64_t(num_heads) * head_dim, kv_row = int64_t(num_kv_heads) * head_dim;
    if (!q_out || !q || !key || !value || !k_cache || !v_cache || !slot_mapping ||
        (rotary_dim > 0 && (!cos_sin || !positions || max_position < 1)))
        return PA_ERR_INVALID_ARG;
    if (!aligned16(q_out) || !aligned16(q) || !aligned16(key) || !aligned16(value) ||
        !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(cos_sin) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) ||
        (reinterpret_cast<uintptr_t>(positions) & 7u))
        return PA_ERR_INVALID_ARG;
    if (q_out_stride < q_row || q_stride < q_row || key_stride < kv_row || value_stride < kv_row ||
        ((q_out_stride | q_stride | key_stride | value_stride) & 7) ||
        (q_out == q && q_out_stride != q_stride))
        return PA_ERR_INVALID_ARG;
    p = pa::RopeParams{};
    p.q_out = q_out;
    p.q = q;
    p.key = key;
    p.value = value;
    p.q_out_stride = q_out_stride;
    p.q_stride = q_stride;
    p.key_stride = key_stride;
    p.value_stride = value_stride;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.cos_sin = cos_sin;
    p.positions = positions;
    p.slots = slot_mapping;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.rotary = rotary_dim;
    p.max_position = max_position;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    p.err = device_error_word();
    return p.err ? PA_OK : PA_ERR_CUDA;
}

template <int D, bool kBf16, bool kInterleaved>
cudaError_t launch_rope(const pa::RopeParams &p, cudaStream_t stream)
{
    const int rows = p.num_heads + 2 * p.num_kv_heads;
    const int per_cta = pa::kRopeThreads / (D / 16) * pa::kRopePasses;
    const dim3 grid(unsigned(p.num_tokens), unsigned((rows + per_cta - 1) / per_cta));
    return launch_pdl(pa::rope_and_cache_kernel<D, kBf16, kInterleaved>, grid,
                      dim3(pa::kRopeThreads), 0, stream, p);
}

template <int D, bool kBf16, bool kInterleaved, bool kE4m3>
cudaError_t launch_rope_q8(pa::RopeParams p, cudaStream_t stream)
{
    constexpr int kRows = pa::kRopeThreads / (D / 16) * pa::kRopePasses, kSpan = 2 * 32 / (D / 16);
    p.groups = std::max((p.num_heads + kRows - 1) / kRows, (p.num_kv_heads + kSpan - 1) / kSpan);
    p.scan_blocks = p.num_blocks <= pa::kScanFew * pa::kScanParts ? pa::kScanFew : pa::kScanMany;
    p.scan_ctas = p.num_tokens > 1 ? 1 + (p.num_blocks - 1) / p.scan_blocks : 0;
    const int64_t ctas = int64_t(p.num_tokens) * p.groups + p.scan_ctas;
    if (ctas > INT32_MAX)
        return cudaErrorInvalidValue;
    return launch_pdl(pa::rope_and_cache_q8_kernel<D, kBf16, kInterleaved, kE4m3>, dim3(unsigned(ctas)),
                      dim3(pa::kRopeThreads), size_t(p.scan_blocks) / 8, stream, p);
}

} // namespace

extern "C" {

pa_status pa_rope_and_cache(void *q_out, int64_t q_out_stride, const void *q, int64_t q_stride,
                            const void *key, int64_t key_stride, const void *value,
                            int64_t value_stride, void *k_cache, void *v_cache,
                            const float *cos_sin, int rotary_dim, int max_position, int interleaved,
                            const int64_t *positions, const int64_t *slot_mapping, int num_tokens,
                            int num_heads, int num_kv_heads, int head_dim, int block_size,
                            int num_blocks, pa_dtype dtype, pa_stream_t stream)
{
    pa::RopeParams p;
    const pa_status st = rope_params(p, q_out, q_out_stride, q, q_stride, key, key_stride, value,
                                     value_stride, k_cache, v_cache, cos_sin, rotary_dim,
                                     max_position, positions, slot_mapping, num_tokens, num_heads,
                                     num_kv_heads, head_dim, block_size, num_blocks, dtype);
    if (st != PA_OK || num_tokens == 0)
        return st;
    const cudaError_t e = with_bool(head_dim == 128, [&](auto d128) {
        return with_bool(dtype == PA_BF16, [&](auto bf16) {
            return with_bool(interleaved != 0, [&](auto inter) {
                return launch_rope<d128 ? 128 : 64, bf16, inter>(
                    p, reinterpret_cast<cudaStream_t>(stream));
            });
        });
    });
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_rope_and_cache_q8(void *q_out, int64_t q_out_stride, const void *q, int64_t q_stride,
                               const void *key, int64_t key_stride, const void *value,
                               int64_t value_stride, void *k_codes, void *v_codes,
                               float *kv_scales, const float *cos_sin, int rotary_dim,
                               int max_position, int interleaved, const int64_t *positions,
                               const int64_t *slot_mapping, int num_tokens, int num_heads,
                               int num_kv_heads, int head_dim, int block_size, int num_blocks,
                               pa_dtype dtype, pa_kv8_type kv_type, pa_stream_t stream)
{
    if (!valid_kv8(kv_type) || (num_tokens > 0 && (!kv_scales || !aligned16(kv_scales))))
        return PA_ERR_INVALID_ARG;
    pa::RopeParams p;
    const pa_status st = rope_params(p, q_out, q_out_stride, q, q_stride, key, key_stride, value,
                                     value_stride, k_codes, v_codes, cos_sin, rotary_dim,
                                     max_position, positions, slot_mapping, num_tokens, num_heads,
                                     num_kv_heads, head_dim, block_size, num_blocks, dtype);
    if (st != PA_OK || num_tokens == 0)
        return st;
    p.kv_scales = reinterpret_cast<float2 *>(kv_scales);
    p.scale_heads = scale_heads(num_kv_heads);
    const cudaError_t e = with_bool(head_dim == 128, [&](auto d128) {
        return with_bool(dtype == PA_BF16, [&](auto bf16) {
            return with_bool(interleaved != 0, [&](auto inter) {
                return with_bool(kv_type == PA_KV8_E4M3, [&](auto e4m3) {
                    return launch_rope_q8<d128 ? 128 : 64, bf16, inter, e4m3>(
                        p, reinterpret_cast<cudaStream_t>(stream));
                });
            });
        });
    });
    return e == cudaSuccess ? PA_OK : e == cudaErrorInvalidValue ? PA_ERR_INVALID_ARG : PA_ERR_CUDA;
}

} // extern "C"
