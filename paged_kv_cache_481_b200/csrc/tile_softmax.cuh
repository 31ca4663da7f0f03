// Softmax of a 128 x 128 score tile held in tensor memory, one row per thread:
// the row in registers, its maximum, and the arithmetic helpers.
#pragma once

#include <cstdint>

#include "tcgen05.cuh"

namespace pa {

constexpr int kScoreCols = 128;   // scores per row of a tile

// ---- softmax arithmetic helpers (inline PTX of documented sm_100 forms) ----

__device__ __forceinline__ float max3f(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 2^x on the special-function unit (approximate, subnormal results flushed).
__device__ __forceinline__ float ex2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One S tile row in registers: all 128 scores of this thread's TMEM lane,
// loaded with one wait.
struct ScoreRow {
    uint32_t s[kScoreCols];
};

__device__ __forceinline__ void load_score_row(uint32_t tS, ScoreRow &r)
{
#pragma unroll
    for (int cc = 0; cc < kScoreCols / 32; ++cc)
        tmem_load32_into(tS + uint32_t(cc * 32), r.s + cc * 32);
    tmem_wait_ld();
}

// Row max of the raw scores; with kMasked only the first `lim` columns count.
template <bool kMasked>
__device__ __forceinline__ float score_row_max(const ScoreRow &r, int lim)
{
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < kScoreCols; i += 8) {
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            float x = __uint_as_float(r.s[i + 2 * a]), y = __uint_as_float(r.s[i + 2 * a + 1]);
            if (kMasked) {
                x = i + 2 * a < lim ? x : -INFINITY;
                y = i + 2 * a + 1 < lim ? y : -INFINITY;
            }
            m[a] = max3f(m[a], x, y);
        }
    }
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

} // namespace pa
