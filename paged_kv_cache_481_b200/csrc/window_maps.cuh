// TMA tensor maps of the window entry points.
#pragma once

#include <algorithm>
#include <cstdint>

#include "tma_host.cuh"

namespace {

// 16-bit values with 128-byte swizzle.  (Copies do not look at the values, so
// the fp16 element type serves bf16 too.)
template <int kDims>
bool swizzled_map(CUtensorMap *map, const void *base, const cuuint64_t (&dims)[kDims],
                  const cuuint64_t (&strides)[kDims - 1], const cuuint32_t (&box)[kDims])
{
    auto encode = tensor_map_encoder();
    cuuint32_t elem[kDims];
    std::fill(elem, elem + kDims, 1u);
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, kDims, const_cast<void *>(base), dims,
                            strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Cache rows of D elements: boxes of `box_rows` rows land as [8-row
// group][64-element half][8 rows][128 bytes].
template <int D>
bool cache_map(CUtensorMap *map, const void *base, uint64_t rows, uint32_t box_rows)
{
    return swizzled_map<4>(map, base, {64, 8, D / 64, rows / 8}, {D * 2, 128, D * 16},
                           {64, 8, D / 64, box_rows / 8});
}

// The memory of an 8-bit cache as 128-byte lines.
inline bool line_map(CUtensorMap *map, const void *base, uint64_t lines, uint32_t box_lines)
{
    return swizzled_map<2>(map, base, {64, lines}, {128}, {64, box_lines});
}

} // namespace
